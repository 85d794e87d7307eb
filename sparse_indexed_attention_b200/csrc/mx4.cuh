// MXFP4 rows of 128 values ([P2] section 5, groups of 32 sharing one scale,
// with E2M1 elements): 64 bytes of codes, element 2i in the low four bits of
// byte i, and 4 E8M0 scale bytes.
//
// One group of 32, largest magnitude m: the scale is 2^e with e = floor(log2 m)
// - 2, so that m / 2^e lies in E2M1's top binade [4, 8), and each element is
// x / 2^e (exact in fp32) rounded to nearest even and saturated at 6.  From
// bf16 the exponent is read off m's bits: e + 127 = max(biased exponent - 2, 0),
// the clamp at -127 covering the subnormals; a zero group takes 127 (2^0).  A
// group with an infinity or NaN takes scale byte 255, E8M0's NaN, and codes 0.
#pragma once
#include <cuda_fp4.h>

#include "dsa_internal.cuh"

namespace dsa {
namespace mx4 {

constexpr int kRowBytes = kDI / 2;  // 64
constexpr int kPieces = 16;         // lanes per row, 8 values each

__device__ __forceinline__ float scale_value(uint32_t byte) {  // 2^(byte - 127); 255 is NaN
  return __uint_as_float(byte == 0u ? 0x00400000u : (byte == 255u ? 0x7FC00000u : byte << 23));
}

// Lane `piece` (of 16 neighbouring lanes) holds values 8 piece .. 8 piece + 7
// of its row; returns their eight codes and the group's scale byte.  Every
// lane of the warp must call it.
__device__ __forceinline__ uint32_t quantize_piece(const uint4& raw, uint32_t* scale_byte) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  // largest |x| as bf16 bits, two values at a time: NaN > infinity > finite in integer order
  uint32_t m = __vmaxu2(__vmaxu2(w[0] & 0x7FFF7FFFu, w[1] & 0x7FFF7FFFu), __vmaxu2(w[2] & 0x7FFF7FFFu, w[3] & 0x7FFF7FFFu));
  m = max(m & 0xFFFFu, m >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const bool finite = m < 0x7F80u;
  const int field = (int)(m >> 7);
  const int byte = m == 0u ? 127 : (field > 2 ? field - 2 : 0);
  *scale_byte = finite ? (uint32_t)byte : 255u;
  // 2^-e = 2^(127 - byte), byte <= 252: a normal number down to 2^-125
  const float inv = __uint_as_float((uint32_t)(254 - byte) << 23);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = make_float2(__uint_as_float(w[i] << 16) * inv, __uint_as_float(w[i] & 0xFFFF0000u) * inv);
    codes |= (uint32_t)__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest) << (8 * i);
  }
  return finite ? codes : 0u;
}

// Lane piece's codes and, from one lane in four, the scale to a row.
__device__ __forceinline__ void store_piece(uint32_t c, uint32_t byte, uint8_t* codes, uint8_t* scales, int64_t row) {
  const int piece = threadIdx.x & (kPieces - 1);
  reinterpret_cast<uint32_t*>(codes + row * kRowBytes)[piece] = c;
  if ((piece & 3) == 0) scales[row * 4 + (piece >> 2)] = (uint8_t)byte;
}

// One row by 16 neighbouring lanes; `live` false computes without storing.
__device__ __forceinline__ void quantize_row(const __nv_bfloat16* __restrict__ src, int64_t src_row, uint8_t* codes,
                                             uint8_t* scales, int64_t dst_row, bool live) {
  const int piece = threadIdx.x & (kPieces - 1);
  uint4 raw = make_uint4(0u, 0u, 0u, 0u);
  if (live) raw = __ldg(reinterpret_cast<const uint4*>(src + src_row * kDI) + piece);
  uint32_t byte;
  const uint32_t c = quantize_piece(raw, &byte);
  if (live) store_piece(c, byte, codes, scales, dst_row);
}

}  // namespace mx4
}  // namespace dsa
