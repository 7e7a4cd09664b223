// fa_packed_bwd.cu — backward pass of attention over packed sequences: the plain kernels, one
// warp a row.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {
namespace {

__device__ __forceinline__ const __nv_bfloat16* row_of(const HeadsView& t, long long i, int h) {
  return static_cast<const __nv_bfloat16*>(t.p) + i * t.token + h * t.head;
}

// The sequence that token i belongs to (-1: none).
__device__ __forceinline__ int sequence_of(const int* cu, int B, int i) {
  if (i < cu[0] || i >= cu[B]) return -1;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

template <int E>
__device__ __forceinline__ void load(const __nv_bfloat16* r, int lane, float (&x)[E]) {
#pragma unroll
  for (int e = 0; e < E; ++e) x[e] = __bfloat162float(r[lane + 32 * e]);
}

template <int E>
__device__ __forceinline__ float dot(const float (&a)[E], const float (&b)[E]) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) s = fmaf(a[e], b[e], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

struct Span {
  int q0, n, k0, m;
};

__device__ __forceinline__ int clamp(int x, int hi) { return min(max(x, 0), hi); }

__device__ __forceinline__ Span span_of(const PackedArgs& a, int b) {
  Span s;
  s.q0 = clamp(a.cu_q[b], a.total_q);
  s.n = max(clamp(a.cu_q[b + 1], a.total_q) - s.q0, 0);
  const int* ck = a.cu_k ? a.cu_k : a.cu_q;
  s.k0 = clamp(ck[b], a.total_k);
  s.m = max(clamp(ck[b + 1], a.total_k) - s.k0, 0);
  return s;
}

__device__ __forceinline__ int keys_of(const PackedArgs& a, const Span& s, int i) {
  return a.causal ? min(max(i + 1 + s.m - s.n, 0), s.m) : s.m;
}

template <int D>
__global__ void fa_packed_dq_kernel(const PackedArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  if (w >= static_cast<long long>(a.total_q) * a.q.heads) return;
  const int i = static_cast<int>(w / a.q.heads), h = static_cast<int>(w % a.q.heads);
  const int b = sequence_of(a.cu_q, a.B, i);
  if (b < 0) return;
  const Span s = span_of(a, b);
  const int keys = keys_of(a, s, i - s.q0), kh = h / (a.q.heads / a.k.heads);
  float q[E], g[E], dq[E], k[E], x[E];
  load(row_of(a.q, i, h), lane, q);
  load(row_of(a.dO, i, h), lane, g);
  load(row_of(a.o, i, h), lane, x);
  const float Di = dot(g, x), lse = a.lse[static_cast<long long>(h) * a.total_q + i];
#pragma unroll
  for (int e = 0; e < E; ++e) dq[e] = 0.0f;
  for (int j = 0; j < keys; ++j) {
    load(row_of(a.k, s.k0 + j, kh), lane, k);
    load(row_of(a.v, s.k0 + j, kh), lane, x);
    const float p = __expf(dot(q, k) * a.scale - lse), ds = p * (dot(g, x) - Di);
#pragma unroll
    for (int e = 0; e < E; ++e) dq[e] = fmaf(ds, k[e], dq[e]);
  }
  __nv_bfloat16* r = const_cast<__nv_bfloat16*>(row_of(a.dq, i, h));
#pragma unroll
  for (int e = 0; e < E; ++e) r[lane + 32 * e] = __float2bfloat16(a.scale * dq[e]);
}

template <int D>
__global__ void fa_packed_dkdv_kernel(const PackedArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32;
  if (w >= static_cast<long long>(a.total_k) * a.k.heads) return;
  const int j = static_cast<int>(w / a.k.heads), kh = static_cast<int>(w % a.k.heads);
  const int b = sequence_of(a.cu_k ? a.cu_k : a.cu_q, a.B, j);
  if (b < 0) return;
  const Span s = span_of(a, b);
  const int G = a.q.heads / a.k.heads;
  float k[E], v[E], dk[E], dv[E], q[E], g[E], x[E];
  load(row_of(a.k, j, kh), lane, k);
  load(row_of(a.v, j, kh), lane, v);
#pragma unroll
  for (int e = 0; e < E; ++e) dk[e] = dv[e] = 0.0f;
  for (int h = kh * G; h < kh * G + G; ++h)
    for (int i = 0; i < s.n; ++i) {
      if (j - s.k0 >= keys_of(a, s, i)) continue;
      load(row_of(a.q, s.q0 + i, h), lane, q);
      load(row_of(a.dO, s.q0 + i, h), lane, g);
      load(row_of(a.o, s.q0 + i, h), lane, x);
      const float lse = a.lse[static_cast<long long>(h) * a.total_q + s.q0 + i];
      const float p = __expf(dot(q, k) * a.scale - lse), ds = p * (dot(g, v) - dot(g, x));
#pragma unroll
      for (int e = 0; e < E; ++e) {
        dv[e] = fmaf(p, g[e], dv[e]);
        dk[e] = fmaf(ds, q[e], dk[e]);
      }
    }
  __nv_bfloat16* rk = const_cast<__nv_bfloat16*>(row_of(a.dk, j, kh));
  __nv_bfloat16* rv = const_cast<__nv_bfloat16*>(row_of(a.dv, j, kh));
#pragma unroll
  for (int e = 0; e < E; ++e) {
    rk[lane + 32 * e] = __float2bfloat16(a.scale * dk[e]);
    rv[lane + 32 * e] = __float2bfloat16(dv[e]);
  }
}

unsigned warps_grid(long long warps) { return static_cast<unsigned>((warps * 32 + 255) / 256); }

}  // namespace

cudaError_t launch_backward_packed(const PackedArgs& a, const CUtensorMap* maps, cudaStream_t s) {
  const unsigned gq = warps_grid(static_cast<long long>(a.total_q) * a.q.heads);
  const unsigned gk = warps_grid(static_cast<long long>(a.total_k) * a.k.heads);
  if (gq > 0) {
    if (a.d == 64) fa_packed_dq_kernel<64><<<gq, 256, 0, s>>>(a);
    else fa_packed_dq_kernel<128><<<gq, 256, 0, s>>>(a);
  }
  if (gk > 0) {
    if (a.d == 64) fa_packed_dkdv_kernel<64><<<gk, 256, 0, s>>>(a);
    else fa_packed_dkdv_kernel<128><<<gk, 256, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace fa
