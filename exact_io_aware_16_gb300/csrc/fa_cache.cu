// fa_cache.cu — the key/value cache: writing new rows (kept in bf16, or
// quantised to e4m3 with a power-of-two scale for each row), reading rows back
// in bf16, and moving the accepted path of a drafted tree into place.
//
// All three are copies with a conversion on the way: every byte is touched once, so
// the calls are bound by HBM for prompts and by launch latency for single tokens.
// A row of d elements belongs to d / 16 lanes, sixteen elements a lane: two 16-byte
// accesses in bf16 and one in e4m3, and a row's maximum takes log2(d / 16) shuffles.
// (Eight elements a lane spent 9 instructions an element on the quantiser, and
// wrote a prompt of 4 x 8 x 8192 rows at 3.9 TB/s.)
//
// Measured (d = 128, e4m3; a plain copy runs at 6.79 TB/s): writing 4 x 8 x 8192 rows
// of keys and values 35 us, 5.8 TB/s (in bf16 43 us, 6.2 TB/s); reading them back
// 33 us, 6.0 TB/s; a token of 8 sequences written 4.1 us, a path of 5 of 16 drafts
// committed for 4 sequences 5 us.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_rows.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

constexpr int kMoveThreads = 256;

// Two bf16 (one word) times s as two e4m3 codes.
__device__ __forceinline__ uint32_t codes2(uint32_t w, float s) {
  return __nv_cvt_float2_to_fp8x2(
      make_float2(__uint_as_float(w << 16) * s, __uint_as_float(w & 0xffff0000u) * s),
      __NV_SATFINITE, __NV_E4M3);
}

// The same where the word may hold infinities, which the saturating conversion
// would make 448: x * 0 turns them into NaN.
__device__ __noinline__ uint32_t codes2_any(uint32_t w, float s) {
  const float lo = __uint_as_float(w << 16), hi = __uint_as_float(w & 0xffff0000u);
  return __nv_cvt_float2_to_fp8x2(
      make_float2(fmaf(lo, 0.0f, lo * s), fmaf(hi, 0.0f, hi * s)), __NV_SATFINITE, __NV_E4M3);
}

// Two e4m3 codes times s as two bf16 (exact: four significant bits).
__device__ __forceinline__ uint32_t values2(uint32_t c, float s) {
  const __half2_raw h =
      __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  return pack_bf16x2(f.x * s, f.y * s);
}

__device__ __forceinline__ uint32_t abs_max(const uint4& x) {
  return __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                  __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}

// 32 bytes at p, in one access where `wide` says that addresses allow it.
__device__ __forceinline__ void store32(uint4* p, bool wide, const uint4& a, const uint4& b) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a.x), "r"(a.y),
                 "r"(a.z), "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    p[0] = a;
    p[1] = b;
  }
}

// Where row r of [B][Hkv][N] lies: its (sequence, head) pair, sequence and index.
struct RowAt {
  int bh, b, i;
  __device__ __forceinline__ RowAt(const CacheMoveArgs& a, int r)
      : bh(a.by_n.divide(r)), b(a.by_heads.divide(bh)), i(r - bh * a.N) {}
};

// Rows run over [B][Hkv][N]; blockIdx.y picks keys or values.  One row a group of D / 16
// lanes: two or four rows in flight a thread gain 2 % on a prompt and lose 1 us where
// there are few rows.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kMoveThreads) fa_cache_write_kernel(const CacheMoveArgs a) {
  constexpr int kLanes = D / 16;
  const bool val = blockIdx.y != 0;
  const int lane = threadIdx.x % kLanes;
  const int r = blockIdx.x * (kMoveThreads / kLanes) + threadIdx.x / kLanes;
  const bool exists = r < a.c.B * a.c.Hkv * a.N;
  const uint4* src = static_cast<const uint4*>(val ? a.in_v : a.in_k) +
                     (static_cast<long long>(r) * kLanes + lane) * 2;
  const uint4 x = exists ? __ldcs(src) : make_uint4(0, 0, 0, 0);
  const uint4 y = exists ? __ldcs(src + 1) : make_uint4(0, 0, 0, 0);
  const RowAt at(a, exists ? r : 0);
  // (lens[b] + i wraps to a position from 2^31 on where it is negative or too large)
  const uint32_t pos = static_cast<uint32_t>(__ldg(a.at + at.b)) + static_cast<uint32_t>(at.i);
  const bool moves = exists && pos < static_cast<uint32_t>(a.c.cap) &&
                     (!a.counts || at.i < __ldg(a.counts + at.b));
  const long long dst = static_cast<long long>(at.bh) * a.c.cap + pos;
  if constexpr (E4M3) {
    uint32_t m = __vmaxu2(abs_max(x), abs_max(y));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m & 0xffffu, m >> 16);
    const bool finite = m < 0x7f80u;
    if (!__all_sync(0xffffffffu, finite)) {  // some row here: over its finite elements
      uint32_t f = __vmaxu2(finite_max8(x), finite_max8(y));
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) f = __vmaxu2(f, __shfl_xor_sync(0xffffffffu, f, o));
      if (!finite) m = max(f & 0xffffu, f >> 16);
    }
    if (!moves) return;
    const int e = scale_exponent(m);
    const float s = pow2_of(-e);
    uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    if (finite) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = codes2(w[i], s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = codes2_any(w[i], s);
    }
    static_cast<uint4*>(val ? a.c.v : a.c.k)[dst * kLanes + lane] =
        make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    if (lane == 0) (val ? a.c.v_scale : a.c.k_scale)[dst] = static_cast<uint8_t>(e + 127);
  } else if (moves) {
    store32(static_cast<uint4*>(val ? a.c.v : a.c.k) + (dst * kLanes + lane) * 2, a.wide, x, y);
  }
}

// The inverse, with zeros in rows that are not read: one row a group of D / 16 lanes.
// Two thirds of the bytes are stores, so that more rows in flight a thread gain
// nothing (4 x 8 x 8192 rows of keys and values in e4m3: 33 us with one row, 34.7
// with two, 34.9 with four), but stores of whole 32-byte sectors do: two rows and two
// stores of 16 bytes took 36.9 us.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kMoveThreads) fa_cache_read_kernel(const CacheMoveArgs a) {
  constexpr int kLanes = D / 16;
  const bool val = blockIdx.y != 0;
  const int lane = threadIdx.x % kLanes;
  const int r = blockIdx.x * (kMoveThreads / kLanes) + threadIdx.x / kLanes;
  if (r >= a.c.B * a.c.Hkv * a.N) return;
  const RowAt at(a, r);
  const long long pos = static_cast<long long>(a.at ? __ldg(a.at + at.b) : 0) + at.i;
  uint4 x = make_uint4(0, 0, 0, 0), y = x;
  if (at.i < __ldg(a.counts + at.b) && pos >= 0 && pos < a.c.cap) {
    const long long row = static_cast<long long>(at.bh) * a.c.cap + pos;
    const uint4* in = static_cast<const uint4*>(val ? a.c.v : a.c.k);
    if constexpr (E4M3) {
      const float f = pow2_of(static_cast<int>((val ? a.c.v_scale : a.c.k_scale)[row]) - 127);
      const uint4 c = in[row * kLanes + lane];
      x = make_uint4(values2(c.x & 0xffffu, f), values2(c.x >> 16, f),
                     values2(c.y & 0xffffu, f), values2(c.y >> 16, f));
      y = make_uint4(values2(c.z & 0xffffu, f), values2(c.z >> 16, f),
                     values2(c.w & 0xffffu, f), values2(c.w >> 16, f));
    } else {
      const uint4* from = in + (row * kLanes + lane) * 2;
      x = from[0];
      y = from[1];
    }
  }
  store32(static_cast<uint4*>(val ? a.out_v : a.out_k) + (static_cast<long long>(r) * kLanes + lane) * 2,
          a.wide, x, y);
}

// One cluster of kCommitCtas CTAs a sequence; its CTAs share the (head, tensor)
// pairs.  A pair's rows (at most 64 of at most 256 bytes) pass through
// registers: all are read, then all are written.  The cluster barrier lies
// between the last read of lens[b] and the write of new_lens[b], which may be
// the same word.
constexpr int kCommitCtas = 8;

template <int ROW_BYTES, bool E4M3>
__global__ void __launch_bounds__(kMoveThreads) __cluster_dims__(kCommitCtas, 1, 1)
    fa_cache_commit_kernel(const CacheMoveArgs a) {
  constexpr int kLanes = ROW_BYTES / 16;
  constexpr int kGroups = kMoveThreads / kLanes;
  constexpr int kSteps = FA_TREE_MAX_DRAFTS / kGroups > 0 ? FA_TREE_MAX_DRAFTS / kGroups : 1;
  const int b = blockIdx.x / kCommitCtas, rank = blockIdx.x % kCommitCtas;
  const int len = a.at[b];
  const int n = min(max(a.counts[b], 0), a.N);
  const bool valid = len >= 0 && len <= a.c.cap;
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  const int lane = threadIdx.x % kLanes;
  const int group = threadIdx.x / kLanes;
  if (valid && n > 0) {
    // source and destination of this thread's rows (-1: the row stays)
    int src[kSteps], src_s = -1;
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const int i = group + u * kGroups;
      src[u] = -1;
      if (i < n && i < a.c.cap - len) {
        const int p = a.path[static_cast<long long>(b) * a.N + i];
        if (p >= 0 && p < a.N && p < a.c.cap - len) src[u] = len + p;
      }
    }
    if (E4M3 && static_cast<int>(threadIdx.x) < n && static_cast<int>(threadIdx.x) < a.c.cap - len) {
      const int p = a.path[static_cast<long long>(b) * a.N + threadIdx.x];
      if (p >= 0 && p < a.N && p < a.c.cap - len) src_s = len + p;
    }
    for (int unit = rank; unit < 2 * a.c.Hkv; unit += kCommitCtas) {
      const long long base =
          (static_cast<long long>(b) * a.c.Hkv + unit / 2) * a.c.cap;
      uint4* rows = static_cast<uint4*>((unit & 1) ? a.c.v : a.c.k) + base * kLanes;
      uint8_t* scale = (E4M3 ? ((unit & 1) ? a.c.v_scale : a.c.k_scale) + base : nullptr);
      uint4 x[kSteps];
      uint8_t s = 0;
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
        if (src[u] >= 0) x[u] = rows[static_cast<long long>(src[u]) * kLanes + lane];
      if (E4M3 && src_s >= 0) s = scale[src_s];
      __syncthreads();
#pragma unroll
      for (int u = 0; u < kSteps; ++u)
        if (src[u] >= 0)
          rows[static_cast<long long>(len + group + u * kGroups) * kLanes + lane] = x[u];
      if (E4M3 && src_s >= 0) scale[len + static_cast<int>(threadIdx.x)] = s;
    }
  }
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  if (rank == 0 && threadIdx.x == 0) a.new_lens[b] = valid ? min(len + min(n, a.c.cap), a.c.cap) : len;
}

bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <int D>
dim3 move_grid(const CacheMoveArgs& a) {
  constexpr long long per = kMoveThreads / (D / 16);
  const long long rows = static_cast<long long>(a.c.B) * a.c.Hkv * a.N;
  return dim3(static_cast<unsigned>((rows + per - 1) / per), 2, 1);
}

}  // namespace

cudaError_t launch_cache_write(const CacheMoveArgs& args, cudaStream_t s) {
  CacheMoveArgs a = args;
  a.by_n = FastDivide(a.N);
  a.by_heads = FastDivide(a.c.Hkv);
  a.wide = aligned32(a.c.k) && aligned32(a.c.v);
  const bool f8 = a.c.format == FA_CACHE_E4M3;
  if (a.c.d == 64) {
    if (f8)
      fa_cache_write_kernel<64, true><<<move_grid<64>(a), kMoveThreads, 0, s>>>(a);
    else
      fa_cache_write_kernel<64, false><<<move_grid<64>(a), kMoveThreads, 0, s>>>(a);
  } else {
    if (f8)
      fa_cache_write_kernel<128, true><<<move_grid<128>(a), kMoveThreads, 0, s>>>(a);
    else
      fa_cache_write_kernel<128, false><<<move_grid<128>(a), kMoveThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheMoveArgs& args, cudaStream_t s) {
  CacheMoveArgs a = args;
  a.by_n = FastDivide(a.N);
  a.by_heads = FastDivide(a.c.Hkv);
  a.wide = aligned32(a.out_k) && aligned32(a.out_v);
  const bool f8 = a.c.format == FA_CACHE_E4M3;
  if (a.c.d == 64) {
    if (f8)
      fa_cache_read_kernel<64, true><<<move_grid<64>(a), kMoveThreads, 0, s>>>(a);
    else
      fa_cache_read_kernel<64, false><<<move_grid<64>(a), kMoveThreads, 0, s>>>(a);
  } else {
    if (f8)
      fa_cache_read_kernel<128, true><<<move_grid<128>(a), kMoveThreads, 0, s>>>(a);
    else
      fa_cache_read_kernel<128, false><<<move_grid<128>(a), kMoveThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

cudaError_t launch_cache_commit(const CacheMoveArgs& a, cudaStream_t s) {
  if (static_cast<long long>(a.c.B) * kCommitCtas > 0x7fffffffll) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(a.c.B) * kCommitCtas;
  if (a.c.format == FA_CACHE_E4M3) {
    if (a.c.d == 64)
      fa_cache_commit_kernel<64, true><<<grid, kMoveThreads, 0, s>>>(a);
    else
      fa_cache_commit_kernel<128, true><<<grid, kMoveThreads, 0, s>>>(a);
  } else {
    if (a.c.d == 64)
      fa_cache_commit_kernel<128, false><<<grid, kMoveThreads, 0, s>>>(a);
    else
      fa_cache_commit_kernel<256, false><<<grid, kMoveThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace fa
