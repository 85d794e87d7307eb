// The FP8 latent cache's device-side decoding ([P2] section 5 table, "Main
// attention KV cache"): E4M3 codes times one power of two per 128 values.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace dsa {

// 8 bytes from global memory through the read-only path.
__device__ __forceinline__ uint2 ld_nc_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// 2^(byte - 127) for a tile-scale byte, exact (2^-127 is the subnormal 0x00400000).
__device__ __forceinline__ float tile_scale(uint32_t byte) {
  return byte == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(byte << 23);
}

// Eight E4M3 codes (little-endian: element k in byte k) times a power-of-two
// scale, as eight bf16 (element 2i in the low half of word i).  Exact: an
// E4M3 value is an fp16 value, and times 2^e it has at most 4 significant bits.
__device__ __forceinline__ uint4 e4m3x8_to_bf16x8(uint2 codes, float sc) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? codes.x : codes.y;
    const __nv_fp8x2_storage_t pair = (__nv_fp8x2_storage_t)((w >> (16 * (i & 1))) & 0xFFFFu);
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(pair, __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * sc, f.y * sc);
    o[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 2^x from the MUFU unit (approximate, subnormal results flushed to 0;
// ex2(-inf) = +0).
__device__ __forceinline__ float ex2_ftz(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace dsa
