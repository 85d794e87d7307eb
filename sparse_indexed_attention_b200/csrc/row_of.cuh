// Which row of a run of equal rows an element belongs to.
// Plain C++ too: the host can run it.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define DSA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DSA_HOST_DEVICE inline
#endif

namespace dsa {

// Division by the length nv of a row as floor((i + add) magic / 2^32): either
//   magic = ceil(2^32 / nv),  add = 0:  right while i e < 2^32, with magic nv = 2^32 + e, or
//   magic = floor(2^32 / nv), add = 1:  right while (i + 1) d <= 2^32, with magic nv = 2^32 - d
// (the first exceeds i / nv by i e / (2^32 nv), which must stay below 1 / nv; the second falls short
// of (i + 1) / nv by (i + 1) d / (2^32 nv), which may be 1 / nv at most).  e + d = nv, so the smaller is
// at most nv / 2: right for i below 2^33 / nv.  The ceiling alone goes wrong in blocks of 32 rows of
// more than 11,585 elements.
struct RowDivisor {
  uint32_t nv, magic, add;  // nv = 1: no product
};

inline RowDivisor row_divisor(uint32_t nv) {
  if (nv == 1) return {1u, 0u, 0u};
  const uint64_t one = 1ull << 32, down = one / nv, d = one % nv;
  return 2 * d < nv && d ? RowDivisor{nv, (uint32_t)down, 1u}
                         : RowDivisor{nv, (uint32_t)(down + (d ? 1 : 0)), 0u};
}

struct RowColumn {
  uint32_t row, column;
};

DSA_HOST_DEVICE RowColumn row_of(uint32_t i, const RowDivisor& by) {
  const uint32_t row = by.nv == 1 ? i : (uint32_t)(((uint64_t)(i + by.add) * by.magic) >> 32);
  return {row, i - row * by.nv};
}

}  // namespace dsa
