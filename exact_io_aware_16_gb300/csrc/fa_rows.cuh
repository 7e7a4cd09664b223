// fa_rows.cuh — the power-of-two scale of an e4m3 row, shared by the cache
// writer and the tree decode's query rows.
#pragma once

#include <cstdint>

#include "fa_internal.h"

namespace fa {

// Scale exponent of a row whose largest finite |x| has the bf16 bits `a`: the
// least e with max|x| 2^-e <= 448 = 1.75 * 2^8, within -100 .. 119.
__device__ __forceinline__ int scale_exponent(uint32_t a) {
  const int e = static_cast<int>(a >> 7) - 135 + ((a & 0x7fu) > 0x60u ? 1 : 0);
  return min(max(e, kScaleExpMin), kScaleExpMax);
}

__device__ __forceinline__ float pow2_of(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Largest finite magnitude of eight bf16, as bf16 bits in both halves' maximum.
__device__ __forceinline__ uint32_t finite_max8(const uint4& x) {
  uint32_t m = 0;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7fff7fffu;
    m = __vmaxu2(m, a & ~__vcmpgeu2(a, 0x7f807f80u));
  }
  return m;
}

}  // namespace fa
