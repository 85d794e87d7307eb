// The MXFP4 index cache's writers and reader (format: mx4.cuh): queries to
// codes, new index keys into the paged cache, and codes back to values.
//
// Each is one pass over its data, bound by HBM: 16 lanes take a row of 128
// values, 16 bytes per lane on the bf16 side, 4 on the code side, so that a
// warp's accesses are whole 128-byte lines and the group maximum is two
// shuffles.
#include <cuda_fp16.h>

#include "mx4.cuh"

namespace dsa {

namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerBlock = kThreads / mx4::kPieces;

__global__ void __launch_bounds__(kThreads)
k_quantize_index_query_mx4(const __nv_bfloat16* __restrict__ qI, int64_t rows, uint8_t* __restrict__ codes,
                           uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + threadIdx.x / mx4::kPieces;
  mx4::quantize_row(qI, row, codes, scales, row, row < rows);
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
  const int64_t row = (int64_t)blockIdx.x * kRowsPerBlock + threadIdx.x / mx4::kPieces;
  if (row >= rows) return;
  const int piece = threadIdx.x & (mx4::kPieces - 1);
  const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(codes + row * mx4::kRowBytes) + piece);
  const float sc = mx4::scale_value(__ldg(scales + row * 4 + (piece >> 2)));
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)((c >> (8 * i)) & 0xFFu), __NV_E2M1);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * sc, f.y * sc);
    o[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  reinterpret_cast<uint4*>(out + row * kDI)[piece] = make_uint4(o[0], o[1], o[2], o[3]);
}

unsigned blocks_for(int64_t rows) { return (unsigned)((rows + kRowsPerBlock - 1) / kRowsPerBlock); }

}  // namespace

cudaError_t launch_quantize_index_query_mx4(const __nv_bfloat16* qI, int T, uint8_t* codes, uint8_t* scales,
                                            cudaStream_t st) {
  const int64_t rows = (int64_t)T * kHI;
  cudaError_t e = launch_pdl("quantize_index_query_mx4", k_quantize_index_query_mx4, dim3(blocks_for(rows)),
                             dim3(kThreads), 0, st, qI, rows, codes, scales);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

cudaError_t launch_append_index_keys_mx4(const SeqsDev& s, const __nv_bfloat16* k, uint8_t* codes, uint8_t* scales,
                                         uint32_t* err, cudaStream_t st) {
  cudaError_t e = launch_pdl("append_index_keys_mx4", k_append_index_keys_mx4, dim3(blocks_for(s.num_tokens)),
                             dim3(kThreads), 0, st, s, k, codes, scales, err);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

cudaError_t launch_dequantize_mx4(const uint8_t* codes, const uint8_t* scales, int64_t rows, __nv_bfloat16* out,
                                  cudaStream_t st) {
  cudaError_t e = launch_pdl("dequantize_mx4", k_dequantize_mx4, dim3(blocks_for(rows)), dim3(kThreads), 0, st, codes,
                             scales, rows, out);
  if (e != cudaSuccess) return e;
  return counted(cudaGetLastError());
}

}  // namespace dsa
