// The part of the Python binding that runs on every call, in native code: the
// tensor checks' fast path, output allocation, and the calls into the library.
//
// A small call (a decode step's rotation, appended keys, a few scores) is bound
// by the host: of 10.5 us per dsa_rope call 5.4 were checks and allocation in
// Python and 1.7 ctypes' conversion of 17 arguments; the launch itself is 3.
// What says why a tensor is refused stays in Python: the functions here decide
// that an argument fits, or hand it to the Python function set by refusals().
//
// The module (_binding) holds
//   refusals(refuse, refuse_seqs)         what raises for need and need_seqs
//   cuda_device(t, name) -> torch.device
//   need(t, name, dtypes, shape, device, min_rows = 0)
//   need_seqs(seqs, device)
//   workspace_size(op, seqs, K, H) -> bytes
//   rows(t, dtype, device) -> (T, H, D, token stride, head stride) or None
//   pools(list, pages, device) -> (bytes of dsa_pool_t[], new pages) or None
//   empty(shape, dtype, device) -> tensor
//   stream_of(device) -> the current stream's address, or None while it captures
// and every asynchronous entry point under its C name, called as
//   dsa_x(device, arguments without the stream) -> status
// which makes `device` current, appends its current stream and releases the GIL.
// Host threads that call on one stream do so in turn.
// A pointer argument is a tensor, None or an address; dsa_seqs_t a Seqs.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAException.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Device.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <limits>
#include <mutex>
#include <string>
#include <tuple>
#include <type_traits>
#include <utility>

#include "dsa.h"

namespace {

const at::Tensor* tensor_of(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// A strided contiguous tensor on `device`.
bool plain(const at::Tensor& t, const at::Device& device) {
  return t.layout() == at::kStrided && t.device() == device && t.is_contiguous();
}

bool fits_one(PyObject* o, PyObject* dtypes, PyObject* shape, const at::Device& device, int64_t min_rows) {
  const at::Tensor* t = tensor_of(o);
  if (!t || !PyTuple_Check(dtypes) || !PyTuple_Check(shape) || !plain(*t, device)) return false;
  bool known = false;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(dtypes); ++i) {
    PyObject* d = PyTuple_GET_ITEM(dtypes, i);
    known = known || (THPDtype_Check(d) && reinterpret_cast<THPDtype*>(d)->scalar_type == t->scalar_type());
  }
  if (!known || t->dim() != PyTuple_GET_SIZE(shape)) return false;
  for (int64_t i = 0; i < t->dim(); ++i) {
    PyObject* w = PyTuple_GET_ITEM(shape, i);
    if (w == Py_None) continue;
    const long long want = PyLong_AsLongLong(w);  // (any integer type)
    if (want != t->size(i)) {
      PyErr_Clear();
      return false;
    }
  }
  return min_rows == 0 || (t->dim() > 0 && t->size(0) >= min_rows);
}

bool device_of(PyObject* o, at::Device& device) {
  if (!THPDevice_Check(o)) {
    PyErr_SetString(PyExc_TypeError, "expected a torch.device");
    return false;
  }
  device = reinterpret_cast<THPDevice*>(o)->device;
  return true;
}

bool count(const char* name, Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "%s: %zd arguments, expected %zd", name, n, want);
  return false;
}

PyObject *refuse = nullptr, *refuse_seqs = nullptr;

PyObject* refusals(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (!count("refusals", n, 2)) return nullptr;
  Py_INCREF(a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(refuse, a[0]);
  Py_XSETREF(refuse_seqs, a[1]);
  Py_RETURN_NONE;
}

// The Python function raises; if it finds nothing wrong, this does.
PyObject* refused(PyObject* f, PyObject* const* a, Py_ssize_t n, const char* what) {
  PyObject* r = f ? PyObject_Vectorcall(f, a, n, nullptr) : nullptr;
  Py_XDECREF(r);
  if (!PyErr_Occurred()) PyErr_Format(PyExc_ValueError, "%s: a tensor that the kernels cannot read", what);
  return nullptr;
}

PyObject* cuda_device(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count("cuda_device", n, 2)) return nullptr;
  const at::Tensor* t = tensor_of(a[0]);
  if (t && t->is_cuda()) return THPDevice_New(t->device());
  PyErr_Format(PyExc_TypeError, "%S: expected a CUDA tensor", a[1]);
  return nullptr;
  END_HANDLE_TH_ERRORS
}

PyObject* need(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Device device(at::kCPU);
  if (n != 5 && !count("need", n, 6)) return nullptr;
  if (!device_of(a[4], device)) return nullptr;
  const long long min_rows = n == 6 ? PyLong_AsLongLong(a[5]) : 0;
  if (min_rows == -1 && PyErr_Occurred()) return nullptr;
  if (fits_one(a[0], a[2], a[3], device, min_rows)) Py_RETURN_NONE;
  PyObject* zero = n == 6 ? nullptr : PyLong_FromLong(0);
  PyObject* args[6] = {a[0], a[1], a[2], a[3], a[4], n == 6 ? a[5] : zero};
  PyObject* r = refused(refuse, args, 6, "need");
  Py_XDECREF(zero);
  return r;
  END_HANDLE_TH_ERRORS
}

// Names of a Seqs' fields, interned once.
struct Names {
  PyObject *q_seq_start, *ctx_len, *page_table, *num_phys_pages, *max_ctx, *num_q_tokens;
} names;

// A Seqs' fields, held for the duration of a call.
struct Fields {
  PyObject *qs = nullptr, *cl = nullptr, *pt = nullptr;
  const at::Tensor *q_seq_start = nullptr, *ctx_len = nullptr, *page_table = nullptr;

  bool read(PyObject* seqs) {
    qs = PyObject_GetAttr(seqs, names.q_seq_start);
    cl = qs ? PyObject_GetAttr(seqs, names.ctx_len) : nullptr;
    pt = cl ? PyObject_GetAttr(seqs, names.page_table) : nullptr;
    if (!pt) return false;
    q_seq_start = tensor_of(qs), ctx_len = tensor_of(cl), page_table = tensor_of(pt);
    return true;
  }
  Fields() = default;
  Fields(const Fields&) = delete;
  ~Fields() {
    Py_XDECREF(qs);
    Py_XDECREF(cl);
    Py_XDECREF(pt);
  }
};

bool fits_seqs(PyObject* seqs, const at::Device& device) {
  Fields f;
  if (!f.read(seqs)) return false;
  for (const at::Tensor* t : {f.q_seq_start, f.ctx_len, f.page_table})
    if (!t || t->scalar_type() != at::kInt || !plain(*t, device)) return false;
  return f.ctx_len->dim() == 1 && f.q_seq_start->dim() == 1 && f.page_table->dim() == 2 &&
         f.q_seq_start->size(0) == f.ctx_len->size(0) + 1 && f.page_table->size(0) == f.ctx_len->size(0);
}

PyObject* need_seqs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Device device(at::kCPU);
  if (!count("need_seqs", n, 2) || !device_of(a[1], device)) return nullptr;
  if (fits_seqs(a[0], device)) Py_RETURN_NONE;
  PyErr_Clear();
  return refused(refuse_seqs, a, 2, "seqs");
  END_HANDLE_TH_ERRORS
}

PyObject* rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Device device(at::kCPU);
  if (!count("rows", n, 3) || !device_of(a[2], device)) return nullptr;
  const at::Tensor* t = tensor_of(a[0]);
  if (!t || t->layout() != at::kStrided || t->device() != device || !THPDtype_Check(a[1]) ||
      reinterpret_cast<THPDtype*>(a[1])->scalar_type != t->scalar_type() || (t->dim() != 2 && t->dim() != 3))
    Py_RETURN_NONE;
  const bool heads = t->dim() == 3;
  const int64_t T = t->size(0), H = heads ? t->size(1) : 1, D = t->size(heads ? 2 : 1);
  if (H < 1 || D < 1 || (t->stride(heads ? 2 : 1) != 1 && D > 1)) Py_RETURN_NONE;
  const int64_t token = T > 1 ? t->stride(0) : 0, head = H > 1 ? t->stride(1) : 0;
  return Py_BuildValue("LLLLL", (long long)T, (long long)H, (long long)D, (long long)token, (long long)head);
  END_HANDLE_TH_ERRORS
}

PyObject* pools(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Device device(at::kCPU);
  if (!count("pools", n, 3) || !device_of(a[2], device)) return nullptr;
  const long long pages = PyLong_AsLongLong(a[1]);
  if (pages == -1 && PyErr_Occurred()) return nullptr;
  if (!PyList_Check(a[0]) && !PyTuple_Check(a[0])) Py_RETURN_NONE;
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[0]);
  if (count > DSA_MAX_POOLS) Py_RETURN_NONE;
  dsa_pool_t out[DSA_MAX_POOLS] = {};
  long long new_pages = pages;
  for (Py_ssize_t i = 0; i < count; ++i) {
    PyObject *p = PySequence_Fast_GET_ITEM(a[0], i), *q = p;
    if (PyTuple_Check(p) || PyList_Check(p)) {
      if (PySequence_Fast_GET_SIZE(p) != 2) Py_RETURN_NONE;
      q = PySequence_Fast_GET_ITEM(p, 1);
      p = PySequence_Fast_GET_ITEM(p, 0);
    }
    const at::Tensor *src = tensor_of(p), *dst = tensor_of(q);
    if (!src || !dst || !plain(*src, device) || src->dim() < 1 || src->size(0) < pages * 64) Py_RETURN_NONE;
    long long here = pages;
    if (p != q) {
      if (!plain(*dst, device) || dst->scalar_type() != src->scalar_type() || dst->dim() != src->dim() ||
          dst->sizes().slice(1) != src->sizes().slice(1) || dst->size(0) < 64)
        Py_RETURN_NONE;
      here = dst->size(0) / 64;
    }
    new_pages = i == 0 ? here : std::min(new_pages, here);
    const int64_t bytes = src->stride(0) * src->element_size();
    if (bytes > std::numeric_limits<int32_t>::max()) Py_RETURN_NONE;
    out[i].src = src->data_ptr();
    out[i].dst = dst->data_ptr();
    out[i].row_bytes = static_cast<int32_t>(bytes);
  }
  return Py_BuildValue("y#L", reinterpret_cast<const char*>(out),
                       static_cast<Py_ssize_t>(sizeof(dsa_pool_t) * std::max<Py_ssize_t>(count, 1)), new_pages);
  END_HANDLE_TH_ERRORS
}

PyObject* empty(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Device device(at::kCPU);
  if (!count("empty", n, 3) || !device_of(a[2], device)) return nullptr;
  if (!PyTuple_Check(a[0]) || !THPDtype_Check(a[1])) {
    PyErr_SetString(PyExc_TypeError, "empty: expected (tuple, torch.dtype, torch.device)");
    return nullptr;
  }
  c10::SmallVector<int64_t, 6> sizes;
  for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[0]); ++i) {
    const long long s = PyLong_AsLongLong(PyTuple_GET_ITEM(a[0], i));
    if (s == -1 && PyErr_Occurred()) return nullptr;
    sizes.push_back(s);
  }
  const auto options = at::TensorOptions().dtype(reinterpret_cast<THPDtype*>(a[1])->scalar_type).device(device);
  return THPVariable_Wrap(at::empty(sizes, options));
  END_HANDLE_TH_ERRORS
}

PyObject* stream_of(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  at::Device device(at::kCPU);
  if (!count("stream_of", n, 1) || !device_of(a[0], device)) return nullptr;
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  C10_CUDA_CHECK(cudaStreamIsCapturing(stream, &status));
  if (status != cudaStreamCaptureStatusNone) Py_RETURN_NONE;
  return PyLong_FromVoidPtr(stream);
  END_HANDLE_TH_ERRORS
}

// One argument of a call, converted from its Python object.
template <class T, class = void>
struct Arg;

template <class T>
struct Arg<T, std::enable_if_t<std::is_integral_v<T>>> {
  T value{};
  bool read(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) return false;
    if constexpr (sizeof(T) < sizeof(long long)) {
      if (v < static_cast<long long>(std::numeric_limits<T>::min()) ||
          v > static_cast<long long>(std::numeric_limits<T>::max())) {
        PyErr_Format(PyExc_OverflowError, "%lld does not fit the argument's %zu bytes", v, sizeof(T));
        return false;
      }
    } else if (std::is_unsigned_v<T> && v < 0) {
      PyErr_Format(PyExc_OverflowError, "%lld is negative", v);
      return false;
    }
    value = static_cast<T>(v);
    return true;
  }
};

template <class T>
struct Arg<T, std::enable_if_t<std::is_enum_v<T>>> {
  T value{};
  bool read(PyObject* o) {
    Arg<int> v;
    if (!v.read(o)) return false;
    value = static_cast<T>(v.value);
    return true;
  }
};

template <>
struct Arg<float> {
  float value = 0.f;
  bool read(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) return false;
    value = static_cast<float>(v);
    return true;
  }
};

template <class T>
struct Arg<T*> {
  T* value = nullptr;
  bool read(PyObject* o) {
    if (o == Py_None) return true;
    if (const at::Tensor* t = tensor_of(o)) {
      value = static_cast<T*>(t->data_ptr());
      return true;
    }
    if (PyLong_Check(o)) {
      value = static_cast<T*>(PyLong_AsVoidPtr(o));
      return value || !PyErr_Occurred();
    }
    if constexpr (std::is_same_v<T, const dsa_pool_t>) {
      if (PyBytes_Check(o)) {
        value = reinterpret_cast<T*>(PyBytes_AS_STRING(o));
        return true;
      }
    }
    PyErr_Format(PyExc_TypeError, "expected a tensor, an address or None, got %s", Py_TYPE(o)->tp_name);
    return false;
  }
};

template <>
struct Arg<const dsa_seqs_t*> {
  dsa_seqs_t seqs{};
  const dsa_seqs_t* value = &seqs;
  Fields f;

  static bool number(PyObject* o, PyObject* name, int32_t& out) {
    PyObject* v = PyObject_GetAttr(o, name);
    Arg<int32_t> a;
    const bool ok = v && a.read(v);
    Py_XDECREF(v);
    out = a.value;
    return ok;
  }
  bool read(PyObject* o) {
    if (!f.read(o)) return false;
    if (!f.q_seq_start || !f.ctx_len || !f.page_table || f.ctx_len->dim() != 1 || f.page_table->dim() != 2) {
      PyErr_SetString(PyExc_TypeError, "expected a Seqs");
      return false;
    }
    seqs.batch = static_cast<int32_t>(f.ctx_len->size(0));
    seqs.page_size = 64;
    seqs.max_pages = static_cast<int32_t>(f.page_table->size(1));
    seqs.q_seq_start = static_cast<const int32_t*>(f.q_seq_start->data_ptr());
    seqs.ctx_len = static_cast<const int32_t*>(f.ctx_len->data_ptr());
    seqs.page_table = static_cast<const int32_t*>(f.page_table->data_ptr());
    return number(o, names.num_q_tokens, seqs.num_q_tokens) && number(o, names.num_phys_pages, seqs.num_phys_pages) &&
           number(o, names.max_ctx, seqs.max_ctx);
  }
};

PyObject* workspace_size(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  Arg<int> op, K, H;
  Arg<const dsa_seqs_t*> seqs;
  if (!count("workspace_size", n, 4) || !op.read(a[0]) || !seqs.read(a[1]) || !K.read(a[2]) || !H.read(a[3]))
    return nullptr;
  return PyLong_FromSize_t(dsa_workspace_size(static_cast<dsa_op_t>(op.value), seqs.value, K.value, H.value));
  END_HANDLE_TH_ERRORS
}

// A call may be several launches over one workspace, which a stream's calls share:
// they must not mix with another thread's.  (Streams that fall on one lock wait for
// each other's launches, no more.)
std::mutex& launching_on(dsa_stream_t stream) {
  static std::mutex locks[64];
  return locks[(reinterpret_cast<uintptr_t>(stream) >> 4) % 64];
}

// The last parameter of an entry point, the stream, comes from the device.
template <auto F, class... A, size_t... I>
PyObject* call(std::tuple<Arg<A>...>& args, PyObject* const* a, Py_ssize_t n, std::index_sequence<I...>) {
  constexpr Py_ssize_t given = sizeof...(I);
  at::Device device(at::kCPU);
  if (!count("call", n, given + 1) || !device_of(a[0], device)) return nullptr;
  // Host memory is taken where there is no GPU: the call then runs its host path
  // up to its first launch, which fails (the tests' way to reach that path).
  if (!device.is_cuda() && c10::cuda::device_count() > 0) {
    PyErr_SetString(PyExc_TypeError, "expected a CUDA device");
    return nullptr;
  }
  if (!(std::get<I>(args).read(a[1 + I]) && ...)) return nullptr;
  c10::cuda::OptionalCUDAGuard guard;
  dsa_stream_t stream = nullptr;
  if (device.is_cuda()) {
    guard.set_device(device);
    stream = c10::cuda::getCurrentCUDAStream(device.index()).stream();
  }
  long status;
  Py_BEGIN_ALLOW_THREADS
  {
    std::lock_guard<std::mutex> one(launching_on(stream));
    status = static_cast<long>(F(std::get<I>(args).value..., stream));
  }
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(status);
}

template <auto F, class R, class... A>
PyObject* entry(R (*)(A...), PyObject* const* a, Py_ssize_t n) {
  std::tuple<Arg<A>...> args;
  return call<F, A...>(args, a, n, std::make_index_sequence<sizeof...(A) - 1>());
}

template <auto F>
PyObject* method(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  return entry<F>(F, a, n);
  END_HANDLE_TH_ERRORS
}

#define DSA_METHOD(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
#define DSA_ENTRY(f) DSA_METHOD(#f, &method<&f>)

PyMethodDef methods[] = {
    DSA_METHOD("refusals", &refusals),
    DSA_METHOD("cuda_device", &cuda_device),
    DSA_METHOD("need", &need),
    DSA_METHOD("need_seqs", &need_seqs),
    DSA_METHOD("workspace_size", &workspace_size),
    DSA_METHOD("rows", &rows),
    DSA_METHOD("pools", &pools),
    DSA_METHOD("empty", &empty),
    DSA_METHOD("stream_of", &stream_of),
    DSA_ENTRY(dsa_quantize_index_query),
    DSA_ENTRY(dsa_quantize_index_query_mx),
    DSA_ENTRY(dsa_quantize_index_query_mx4),
    DSA_ENTRY(dsa_append_index_keys_mx4),
    DSA_ENTRY(dsa_dequantize_mx4),
    DSA_ENTRY(dsa_index_scores),
    DSA_ENTRY(dsa_topk),
    DSA_ENTRY(dsa_sparse_mla_fwd_ex),
    DSA_ENTRY(dsa_sparse_mla_fwd_noalloc),
    DSA_ENTRY(dsa_index_topk_attn_ex),
    DSA_ENTRY(dsa_attn_mass),
    DSA_ENTRY(dsa_evict_select),
    DSA_ENTRY(dsa_evict_compact),
    DSA_ENTRY(dsa_rope),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  names.q_seq_start = PyUnicode_InternFromString("q_seq_start");
  names.ctx_len = PyUnicode_InternFromString("ctx_len");
  names.page_table = PyUnicode_InternFromString("page_table");
  names.num_phys_pages = PyUnicode_InternFromString("num_phys_pages");
  names.max_ctx = PyUnicode_InternFromString("max_ctx");
  names.num_q_tokens = PyUnicode_InternFromString("num_q_tokens");
  return PyModule_Create(&module_def);
}
