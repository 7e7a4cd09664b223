// fa_tree.cu — attention of a tree of drafted tokens over the key/value cache
// (bf16 or e4m3), grouped heads, a length for each sequence.
//
// One warp a query row: it walks the keys that the row sees, each lane holding
// d / 32 channels, with the running maximum and sum of the softmax.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kTreeThreads = 128;

template <int D, bool E4M3>
__device__ __forceinline__ void load_row(const void* t, const uint8_t* scale, long long row,
                                         int lane, float (&x)[D / 32]) {
  if (E4M3) {
    const float s = exp2f(static_cast<float>(static_cast<int>(scale[row]) - 127));
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const __half_raw h = __nv_cvt_fp8_to_halfraw(
          static_cast<const uint8_t*>(t)[row * D + lane * (D / 32) + c], __NV_E4M3);
      x[c] = __half2float(__half(h)) * s;
    }
  } else {
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      x[c] = __bfloat162float(
          static_cast<const __nv_bfloat16*>(t)[row * D + lane * (D / 32) + c]);
  }
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kTreeThreads) fa_tree_kernel(const TreeArgs a) {
  constexpr int kC = D / 32;
  const long long row = static_cast<long long>(blockIdx.x) * (kTreeThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (row >= static_cast<long long>(a.c.B) * a.Hq * a.T) return;
  const int t = static_cast<int>(row % a.T);
  const int hq = static_cast<int>(row / a.T % a.Hq);
  const int b = static_cast<int>(row / a.T / a.Hq);
  const long long base = (static_cast<long long>(b) * a.c.Hkv + hq / (a.Hq / a.c.Hkv)) * a.c.cap;
  const int len = min(max(a.lens[b], 0), a.c.cap);
  const unsigned long long seen =
      a.mask ? a.mask[static_cast<long long>(b) * a.mask_stride + t] : (2ull << t) - 1;
  const int end = static_cast<int>(min(static_cast<long long>(a.c.cap), static_cast<long long>(len) + a.T));
  float q[kC], o[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    q[c] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[row * D + lane * kC + c]) * a.scale;
    o[c] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int p = 0; p < end; ++p) {
    if (p >= len && !(seen >> (p - len) & 1)) continue;
    float x[kC], s = 0.0f;
    load_row<D, E4M3>(a.c.k, a.c.k_scale, base + p, lane, x);
#pragma unroll
    for (int c = 0; c < kC; ++c) s = fmaf(q[c], x[c], s);
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    load_row<D, E4M3>(a.c.v, a.c.v_scale, base + p, lane, x);
    const float m_new = fmaxf(m, s);
    const float base_m = m_new == -INFINITY ? 0.0f : m_new;
    const float alpha = expf(m - base_m), pr = expf(s - base_m);
    l = l * alpha + pr;
#pragma unroll
    for (int c = 0; c < kC; ++c) o[c] = fmaf(pr, x[c], o[c] * alpha);
    m = m_new;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int c = 0; c < kC; ++c)
    static_cast<__nv_bfloat16*>(a.o)[row * D + lane * kC + c] =
        __float2bfloat16_rn(l == 0.0f ? 0.0f : o[c] * inv);
  if (lane == 0) a.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

template <int D, bool E4M3>
cudaError_t launch(const TreeArgs& a, cudaStream_t s) {
  const long long rows = static_cast<long long>(a.c.B) * a.Hq * a.T;
  const long long per = kTreeThreads / 32;
  fa_tree_kernel<D, E4M3><<<static_cast<unsigned>((rows + per - 1) / per), kTreeThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_tree(const TreeArgs& a, cudaStream_t s) {
  const bool f8 = a.c.format == FA_CACHE_E4M3;
  if (a.c.d == 64) return f8 ? launch<64, true>(a, s) : launch<64, false>(a, s);
  return f8 ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace fa
