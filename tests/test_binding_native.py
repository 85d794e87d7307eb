"""The native part of the binding: its checks agree with their Python reasons,
and its argument conversions refuse what the library would misread."""
import ctypes

import pytest
import torch

import sparse_indexed_attention_b200 as dsa
from sparse_indexed_attention_b200 import _binding

CPU = torch.device("cpu")
on_host = pytest.mark.skipif(torch.cuda.is_available(), reason="host buffers must not reach a GPU launch")


def test_every_asynchronous_entry_point_is_there():
    """Those whose last argument is the stream, but for the ones that synchronise
    and the short form of an _ex call."""
    rest = {"dsa_check_error", "dsa_check_error_noalloc", "dsa_sparse_mla_fwd", "dsa_index_topk_attn",
            "dsa_workspace_size", "dsa_set_wait_limit_ns", "dsa_status_string", "dsa_launches_in_last_call",
            "dsa_launch_timing", "dsa_last_launch_times"}
    assert {n for n in dir(_binding) if n.startswith("dsa_")} == set(dsa.EXPORTS) - rest


@pytest.mark.parametrize("bad, error, match", [
    (None, TypeError, "torch.Tensor"),
    ([1.0], TypeError, "torch.Tensor"),
    (torch.zeros(4, 3, dtype=torch.float64), TypeError, "dtype"),
    (torch.zeros(4, 4), ValueError, "shape"),
    (torch.zeros(12), ValueError, "shape"),
    (torch.zeros(4, 3, 1), ValueError, "shape"),
    (torch.zeros(3, 4).t(), ValueError, "contiguous"),
    (torch.zeros(8, 3)[::2], ValueError, "contiguous"),
    (torch.zeros(3, 3), ValueError, "at least 4"),
    (torch.zeros(4, 3, device="meta"), ValueError, "meta"),
    (torch.zeros(4, 3).to_sparse(), ValueError, "contiguous"),
])
def test_need(bad, error, match):
    _binding.need(torch.zeros(4, 3), "t", (torch.float16, torch.float32), (None, 3), CPU, 4)
    _binding.need(torch.zeros(0, 3), "t", (torch.float32,), (0, 3), CPU)
    with pytest.raises(error, match=match):
        _binding.need(bad, "t", (torch.float16, torch.float32), (None, 3), CPU, 4)


def test_need_takes_sizes_only():
    import numpy as np
    _binding.need(torch.zeros(4, 3), "t", (torch.float32,), (np.int64(4), np.int32(3)), CPU)
    with pytest.raises(ValueError, match="shape"):
        _binding.need(torch.zeros(4, 3), "t", (torch.float32,), (np.int64(3), 3), CPU)
    with pytest.raises(ValueError, match="shape"):
        _binding.need(torch.zeros(4), "t", (torch.float32,), ("4",), CPU)
    with pytest.raises(ValueError, match="shape"):
        _binding.need(torch.zeros(4), "t", (torch.float32,), (2 ** 70,), CPU)
    with pytest.raises(TypeError):
        _binding.need(torch.zeros(4), "t", (torch.float32,), (4,), "cpu")
    with pytest.raises(TypeError):
        _binding.need(torch.zeros(4), "t", (torch.float32,))


def _seqs(qs=None, cl=None, pt=None, **kw):
    i = torch.int32
    return dsa.Seqs(torch.tensor([0, 1, 2], dtype=i) if qs is None else qs, torch.tensor([5, 6], dtype=i) if cl is None
                    else cl, torch.zeros(2, 3, dtype=i) if pt is None else pt, kw.get("pages", 4), 6, kw.get("T", 2))


def test_need_seqs():
    _binding.need_seqs(_seqs(), CPU)
    i = torch.int32
    for kw, error, match in ((dict(qs=torch.zeros(2, dtype=i)), ValueError, "q_seq_start"),
                             (dict(qs=torch.zeros(3)), TypeError, "q_seq_start"),
                             (dict(cl=torch.zeros(2, dtype=torch.int64)), TypeError, "ctx_len"),
                             (dict(pt=torch.zeros(3, 3, dtype=i)), ValueError, "page_table"),
                             (dict(pt=torch.zeros(2, 6, dtype=i)[:, ::2]), ValueError, "page_table"),
                             (dict(pt=torch.zeros(2, 3, dtype=i, device="meta")), ValueError, "page_table")):
        with pytest.raises(error, match=match):
            _binding.need_seqs(_seqs(**kw), CPU)
    with pytest.raises((TypeError, AttributeError)):
        _binding.need_seqs(None, CPU)


def test_workspace_size_is_the_library_s():
    seqs = _seqs()
    c = seqs.c()
    for op in range(10):
        assert _binding.workspace_size(op, seqs, 128, 16) == dsa.raw().dsa_workspace_size(op, ctypes.byref(c), 128, 16)


def test_rows():
    x = torch.zeros(5, 4, 8)
    assert _binding.rows(x, torch.float32, CPU) == (5, 4, 8, 32, 8)
    assert _binding.rows(x[:, :2, 4:], torch.float32, CPU) == (5, 2, 4, 32, 8)
    assert _binding.rows(x[0], torch.float32, CPU) == (4, 1, 8, 8, 0)
    assert _binding.rows(x[:1, :1], torch.float32, CPU) == (1, 1, 8, 0, 0)
    assert _binding.rows(x[:0], torch.float32, CPU)[:3] == (0, 4, 8)
    for bad in (x[..., ::2], x[:, :0], x[..., :0], x[0, 0], x[None], x.half(), x.to("meta"), None):
        assert _binding.rows(bad, torch.float32, CPU) is None


def test_pools():
    a, b = torch.zeros(256, 8), torch.zeros(128, 8)
    raw, pages = _binding.pools([a, (a, b), (a.byte(), a.byte())], 4, CPU)
    c = (dsa.DsaPoolC * 3).from_buffer_copy(raw)
    assert pages == 2 and [p.row_bytes for p in c] == [32, 32, 8]
    assert (c[0].src, c[0].dst, c[1].dst) == (a.data_ptr(), a.data_ptr(), b.data_ptr())
    assert _binding.pools([], 4, CPU)[1] == 4
    for bad in ([a[:255]], [a, None], [(a, b.byte())], [(a, b[:, :4].contiguous())], [(a, b[:63])], [(a, b, b)],
                [a[:, ::2]], [torch.zeros(())], [a] * 9, [a.to("meta")]):
        assert _binding.pools(bad, 4, CPU) is None


def test_empty():
    t = _binding.empty((2, 0, 3), torch.bfloat16, CPU)
    assert t.shape == (2, 0, 3) and t.dtype == torch.bfloat16 and t.device == CPU
    with pytest.raises(RuntimeError):
        _binding.empty((-2,), torch.bfloat16, CPU)
    with pytest.raises(TypeError):
        _binding.empty([2], torch.bfloat16, CPU)


@on_host
def test_arguments_of_a_call():
    """A call with host memory ends before its first launch; these end sooner."""
    x, s = torch.zeros(4, 64), torch.zeros(4, 4, dtype=torch.uint8)
    f = _binding.dsa_dequantize_mx4
    assert f(CPU, x, s, -1, x) == dsa.DSA_ERR_INVALID_ARG
    assert f(CPU, None, s.data_ptr(), 1, x) == dsa.DSA_ERR_INVALID_ARG
    for args, error in (((CPU, x, s, 1), TypeError), ((CPU, x, s, 1, x, 0), TypeError), (("cpu", x, s, 1, x), TypeError),
                        ((CPU, "x", s, 1, x), TypeError), ((CPU, x, s, 1.5, x), TypeError),
                        ((CPU, x, s, 2 ** 63, x), OverflowError), ((CPU, x, s, b"1", x), TypeError),
                        ((CPU, b"x", s, 1, x), TypeError)):
        with pytest.raises(error):
            f(*args)
    with pytest.raises(OverflowError):
        _binding.dsa_quantize_index_query_mx4(CPU, x, 2 ** 31, x, x)
    with pytest.raises(OverflowError):
        _binding.dsa_append_index_keys_mx4(CPU, _seqs(), x, x, x, x, -1)
    with pytest.raises(OverflowError):
        _binding.dsa_append_index_keys_mx4(CPU, _seqs(T=2 ** 31), x, x, x, x, 256)
    with pytest.raises(TypeError):
        _binding.dsa_append_index_keys_mx4(CPU, _seqs(pt=3), x, x, x, x, 256)
    with pytest.raises((TypeError, AttributeError)):
        _binding.dsa_append_index_keys_mx4(CPU, None, x, x, x, x, 256)


@pytest.mark.gpu
def test_host_memory_is_refused_where_there_is_a_gpu():
    x = torch.zeros(4, 64)
    with pytest.raises(TypeError, match="CUDA"):
        _binding.dsa_dequantize_mx4(CPU, x, x, 1, x)
    with pytest.raises(TypeError, match="codes: expected a CUDA tensor"):
        dsa.dsa_dequantize_mx4(x.byte(), x.byte())


@pytest.mark.gpu
def test_calls_follow_the_current_stream():
    codes = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    scales = torch.full((4, 4), 127, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        codes.fill_(0x22)                # E2M1 1.0 twice
        out = dsa.dsa_dequantize_mx4(codes, scales)
    torch.cuda.current_stream().wait_stream(side)
    assert (out == 1.0).all()


@pytest.mark.gpu
def test_a_captured_workspace_outlives_a_larger_one():
    import weakref
    small = dsa.workspace(1 << 10, "cuda", "outlive")
    ref = weakref.ref(small)
    del small
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert dsa.workspace(1 << 10, "cuda", "outlive") is ref()
        ref().add_(1)
    assert dsa.workspace(1 << 14, "cuda", "outlive").numel() == 1 << 14
    assert ref() is not None
    g.replay()
    torch.cuda.synchronize()
    assert (ref() == 1).all() and not dsa.workspace(1 << 14, "cuda", "outlive").any()
