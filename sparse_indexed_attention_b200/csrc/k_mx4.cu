// The MXFP4 index cache's writers and reader (format: mx4.cuh): queries to
// codes, new index keys into the paged cache, and codes back to values.
//
// Each is one pass over its data, bound by HBM: 16 lanes take a row of 128
// values, 16 bytes per lane on the bf16 side, 4 on the code side, so that a
// warp's accesses are whole 128-byte lines and the group maximum is two
// shuffles.  Four rows per thread group: one row each was bound by the start of
// blocks (4096 x 64 rows: 18.5 us, now 14.6 us for 85 MB, 89 % of the measured copy rate;
// back: 18.1, now 10.4 us, part of it from L2).  Values pass as streaming data (read or
// written once: a chunk's four calls 36.1 -> 32.8 us); the group's maximum is taken
// two values at a time (31.4 us).
#include <cuda_fp16.h>

#include "mx4.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerBlock = kThreads / mx4::kPieces;
constexpr int kBatch = 4;                     // rows per thread group

__global__ void __launch_bounds__(kThreads)
k_quantize_index_query_mx4(const __nv_bfloat16* __restrict__ qI, int64_t rows, uint8_t* __restrict__ codes,
                           uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int64_t row0 = (int64_t)blockIdx.x * (kBatch * kRowsPerBlock) + threadIdx.x / mx4::kPieces;
  const int piece = threadIdx.x & (mx4::kPieces - 1);
  uint4 raw[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int64_t row = row0 + u * kRowsPerBlock;
    raw[u] = row < rows ? __ldcs(reinterpret_cast<const uint4*>(qI + row * kDI) + piece) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int64_t row = row0 + u * kRowsPerBlock;
    uint32_t byte;
    const uint32_t c = mx4::quantize_piece(raw[u], &byte);
    if (row < rows) mx4::store_piece(c, byte, codes, scales, row);
  }
}

// Token t's key into the pool row of its position.
__global__ void __launch_bounds__(kThreads)
k_append_index_keys_mx4(const SeqsDev s, const __nv_bfloat16* __restrict__ k, uint8_t* __restrict__ codes,
                        uint8_t* __restrict__ scales, uint32_t* err) {
  pdl_wait();
  pdl_trigger();
  const int64_t t = (int64_t)blockIdx.x * kRowsPerBlock + threadIdx.x / mx4::kPieces;
  int64_t row = -1;
  if (t < s.num_tokens) {
    const TokenPlace at = locate_token(s, (int)t);
    if (at.pos >= 0)
      row = phys_row(s.page_table, s.max_pages, s.num_phys_pages, at.seq, at.pos, err);
    else
      raise_error(err, kErrBadIndex);
  }
  mx4::quantize_row(k, t, codes, scales, row, row >= 0);
}

// Codes and scales back to bf16, exact: an E2M1 value has two significant
// bits, and the subnormal scales 2^-127, 2^-126 stay within bf16's subnormals.
__global__ void __launch_bounds__(kThreads)
k_dequantize_mx4(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows,
                 __nv_bfloat16* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int64_t row0 = (int64_t)blockIdx.x * (kBatch * kRowsPerBlock) + threadIdx.x / mx4::kPieces;
  const int piece = threadIdx.x & (mx4::kPieces - 1);
  uint32_t c[kBatch], byte[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int64_t row = min(row0 + u * kRowsPerBlock, rows - 1);
    c[u] = __ldg(reinterpret_cast<const uint32_t*>(codes + row * mx4::kRowBytes) + piece);
    byte[u] = __ldg(scales + row * 4 + (piece >> 2));
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    const int64_t row = row0 + u * kRowsPerBlock;
    const float sc = mx4::scale_value(byte[u]);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((c[u] >> (8 * i)) & 0xFFu), __NV_E2M1);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * sc, f.y * sc);
      o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if (row < rows) __stcs(reinterpret_cast<uint4*>(out + row * kDI) + piece, make_uint4(o[0], o[1], o[2], o[3]));
  }
}

unsigned blocks_for(int64_t rows, int batch) {
  const int per = batch * kRowsPerBlock;
  return (unsigned)((rows + per - 1) / per);
}

}  // namespace

cudaError_t launch_quantize_index_query_mx4(const __nv_bfloat16* qI, int T, uint8_t* codes, uint8_t* scales,
                                            cudaStream_t st) {
  const int64_t rows = (int64_t)T * kHI;
  cudaError_t e = launch_pdl("quantize_index_query_mx4", k_quantize_index_query_mx4, dim3(blocks_for(rows, kBatch)),
                             dim3(kThreads), 0, st, qI, rows, codes, scales);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

cudaError_t launch_append_index_keys_mx4(const SeqsDev& s, const __nv_bfloat16* k, uint8_t* codes, uint8_t* scales,
                                         uint32_t* err, cudaStream_t st) {
  cudaError_t e = launch_pdl("append_index_keys_mx4", k_append_index_keys_mx4, dim3(blocks_for(s.num_tokens, 1)),
                             dim3(kThreads), 0, st, s, k, codes, scales, err);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

cudaError_t launch_dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, __nv_bfloat16* out,
                                  cudaStream_t st) {
  cudaError_t e = launch_pdl("dequantize_mx4", k_dequantize_mx4, dim3(blocks_for(rows, kBatch)), dim3(kThreads), 0, st,
                             codes, scales, rows, out);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

}  // namespace dsa
