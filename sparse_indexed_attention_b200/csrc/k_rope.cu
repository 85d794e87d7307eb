// Rotary positions: part of each head's dims turns, pair by pair, by an angle
// that grows with the token's position,
//
//   (a, b) -> m (a cos p f_j - b sin p f_j,  a sin p f_j + b cos p f_j)
//
// for pair j of rot_dim / 2 (dims 2j, 2j+1 interleaved, or j, j + rot_dim/2 in
// the half layout), position p and amplitude m.  The transposed map (sin
// negated) is the gradient and, with m = 1, the inverse.
//
// The angle.  f_j arrives as turns per position in units of 2^-64, so p f_j
// mod one turn is one wrapping 64-bit product: exact for any position, where
// an fp32 (or fp64) product of a far position loses the low bits that the
// sine needs.  The signed fraction, in [-1/2, 1/2) turn, is rounded to fp32
// once (an error of at most 2^-26 turn, 1e-7 rad), so cos and sin are as
// good as fp32 holds them.
//
// What bounds it.  Each value is read and written once: HBM.  cos and sin
// depend on (token, pair) alone, so a block computes them once for its tokens
// into shared memory and its heads share them; computed per value they would
// cost more issue slots than the memory time allows (2 x ~40 instructions per
// pair against 4 bytes moved per bf16 value pair at 44 B/ns per SM).
// 8192 tokens x 64 heads x 128 dims, half of them rotated: 50 us, 82 % of the measured
// copy rate; what is left is latency (each thread has one unit in flight).
// A thread handles 16-byte vectors where base, strides, offset and rot_dim
// allow it, else single elements (slices at odd offsets).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_internal.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxAngles = 2048;  // (token, pair) angles of a block in shared memory (16 KB)

struct RopeArgs {
  const void* x;
  void* out;
  int64_t xt, xh, ot, oh;  // element strides of tokens and heads
  const void* pos;
  const uint64_t* turns;
  float amp;
  int T, H, D, rot, offset;
  int tb, hb;              // tokens and heads per block
  int head_blocks;
  uint32_t units_magic;    // ceil(2^32 / units), or 0: divide
  bool pos64, transpose, copy;  // copy: dims outside the rotated range are written too
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class E> __device__ __forceinline__ E from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

template <class E, int VEC>
struct alignas(sizeof(E) * VEC) Vec {
  E v[VEC];
};

template <class E>
__device__ __forceinline__ void rotate(E& a, E& b, float2 cs) {
  const float p = to_f(a), q = to_f(b);
  a = from_f<E>(fmaf(p, cs.x, -q * cs.y));
  b = from_f<E>(fmaf(p, cs.y, q * cs.x));
}

// Stores 16 bytes as data that this kernel does not read again (8192 tokens x 64
// heads x 128 dims 52.3 -> 51.2 us, 1024 tokens 9.6 -> 8.6).
template <class V>
__device__ __forceinline__ void put(V* p, const V& v) {
  if constexpr (sizeof(V) == 16)
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&v));
  else
    *p = v;
}

// One block: tb tokens x hb heads.  Work units of a (token, head) row: the
// rotated ones first -- VEC consecutive dims interleaved (VEC = 1: one pair), or a
// vector of each half -- then the copied vectors of the other dims.
template <class E, int VEC, bool kHalf>
__global__ void __launch_bounds__(kThreads, 8) k_rope(const RopeArgs a) {
  __shared__ float2 cs[kMaxAngles];
  using V = Vec<E, VEC>;
  const int half = a.rot >> 1;
  const int64_t t0 = (int64_t)(blockIdx.x / a.head_blocks) * a.tb;
  const int h0 = (int)(blockIdx.x % a.head_blocks) * a.hb;
  const int nt = (int)min((int64_t)a.tb, a.T - t0), nh = min(a.hb, a.H - h0);
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int k = i / half, j = i - k * half;
    const int64_t p = a.pos64 ? static_cast<const int64_t*>(a.pos)[t0 + k]
                              : (int64_t) static_cast<const int32_t*>(a.pos)[t0 + k];
    const int64_t frac = (int64_t)((uint64_t)p * a.turns[j]);  // turns mod 1, signed, in units of 2^-64
    float s, c;
    sincospif(__ll2float_rn(frac) * 0x1p-63f, &s, &c);         // angle / pi = 2 * turns
    cs[i] = make_float2(c * a.amp, (a.transpose ? -s : s) * a.amp);
  }
  __syncthreads();
  constexpr int kPairVec = kHalf ? VEC : (VEC > 1 ? VEC / 2 : 1);  // pairs per rotated unit
  const int nrot = half / kPairVec;
  const int units = nrot + (a.copy ? (a.D - a.rot) / VEC : 0);
  const int total = nt * nh * units;
  for (int i = threadIdx.x; i < total; i += kThreads) {
    const int row = a.units_magic ? (int)__umulhi((uint32_t)i, a.units_magic) : i / units, u = i - row * units;
    const int k = row / nh, h = row - k * nh;
    const E* x = static_cast<const E*>(a.x) + (t0 + k) * a.xt + (int64_t)(h0 + h) * a.xh;
    E* o = static_cast<E*>(a.out) + (t0 + k) * a.ot + (int64_t)(h0 + h) * a.oh;
    // copied and rotated units share their loads and stores: apart, a warp that
    // holds both would wait for memory twice
    constexpr bool kTwo = kHalf || VEC == 1;  // a rotated unit is two vectors: the pairs' first and second elements
    const bool turn = u < nrot;
    int d0 = a.offset + (VEC == 1 && !kHalf ? 2 * u : u * VEC);
    if (!turn) {
      d0 = (u - nrot) * VEC;
      if (d0 >= a.offset) d0 += a.rot;
    }
    V va = *reinterpret_cast<const V*>(x + d0), vb;
    if constexpr (kTwo)
      if (turn) vb = *reinterpret_cast<const V*>(x + d0 + (kHalf ? half : 1));
    if (turn) {
      const float2* c = cs + k * half + u * kPairVec;
      if constexpr (kTwo) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) rotate(va.v[e], vb.v[e], c[e]);
        put(reinterpret_cast<V*>(o + d0 + (kHalf ? half : 1)), vb);
      } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) rotate(va.v[2 * e], va.v[2 * e + 1], c[e]);
      }
    }
    put(reinterpret_cast<V*>(o + d0), va);
  }
}

template <class E>
cudaError_t launch_typed(const RopeArgs& a, bool half_layout, bool vec, unsigned grid, cudaStream_t st) {
  constexpr int W = 16 / (int)sizeof(E);
  auto go = [&](auto kernel) { return launch_pdl("rope", kernel, dim3(grid), dim3(kThreads), 0, st, a); };
  if (vec) return half_layout ? go(k_rope<E, W, true>) : go(k_rope<E, W, false>);
  return half_layout ? go(k_rope<E, 1, true>) : go(k_rope<E, 1, false>);
}

}  // namespace

cudaError_t launch_rope(const RopeCall& r, cudaStream_t st) {
  const int size = r.dtype == DSA_ROPE_F32 ? 4 : 2, W = 16 / size;
  RopeArgs a{r.x,   r.out, r.xt,  r.xh,     r.ot, r.oh, r.pos, r.turns, r.amp, r.T, r.H, r.D,
             r.rot, r.offset, 1, r.H, 1, 0u, r.pos64, r.transpose, r.x != r.out};
  auto ok = [&](int64_t v) { return v % W == 0; };
  const bool vec = (reinterpret_cast<uintptr_t>(r.x) | reinterpret_cast<uintptr_t>(r.out)) % 16 == 0 && ok(r.xt) &&
                   ok(r.xh) && ok(r.ot) && ok(r.oh) && ok(r.offset) && ok(r.D) &&
                   ok(r.half_layout ? r.rot / 2 : r.rot);
  // units of a row, and a block's share: about four units per thread where the units
  // fill the GPU's threads, so that a block's angles serve more of them (8192 tokens x 64
  // heads of 64 dims: 27.9 us, 36.6 with one unit), eight where they fill them 16 times
  // (8192 x 64 heads of 128 dims: 49.7 us, 51.2 with four; 2048: 15.7 and 15.4), else
  // one (64 x 128 heads: 2.1 us, 3.1 with four; 256 x 128: 3.7 and 3.5)
  const int lanes = vec ? W : 1;
  const int64_t units = (r.half_layout || !vec ? r.rot / 2 / lanes : r.rot / lanes) + (a.copy ? (r.D - r.rot) / lanes : 0);
  const int64_t all = units * r.H * r.T;
  const int64_t full = (int64_t)148 * 6 * kThreads;
  const int64_t want = (all >= 16 * full ? 8 : all >= full ? 4 : 1) * kThreads;
  if (units * r.H >= want) {
    a.hb = (int)((want + units - 1) / units);
  } else {
    const int64_t t = want / (units * r.H);
    const int64_t most = kMaxAngles / (r.rot / 2);
    a.tb = (int)(t < most ? t : most);
    if (a.tb > r.T) a.tb = r.T;
  }
  // i / units by a product: exact while i units < 2^32 (a block has at most 2048 + units units)
  if (units > 1 && units <= 16384) a.units_magic = (uint32_t)(((1ull << 32) + units - 1) / units);
  a.head_blocks = (r.H + a.hb - 1) / a.hb;
  const int64_t grid = ((int64_t)r.T + a.tb - 1) / a.tb * a.head_blocks;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = r.dtype == DSA_ROPE_F32    ? launch_typed<float>(a, r.half_layout, vec, (unsigned)grid, st)
                  : r.dtype == DSA_ROPE_F16 ? launch_typed<__half>(a, r.half_layout, vec, (unsigned)grid, st)
                                            : launch_typed<__nv_bfloat16>(a, r.half_layout, vec, (unsigned)grid, st);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

}  // namespace dsa
