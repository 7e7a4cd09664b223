// fa_packed_bwd.cu — backward pass of attention over packed sequences with grouped heads.
//
//   P = exp(scale Q K^T - lse),  dP = dO V^T,  D_i = sum_j P_ij dP_ij,  dS = P o (dP - D),
//   dQ = scale dS K,  dK = scale sum_heads dS^T Q,  dV = sum_heads P^T dO.
//
// Two kernels over the tiles of fa_packed.cuh, each bound by the tensor core:
//   * dq: 128 query rows stay while 64-row key and value tiles stream; four products a
//     tile (S, dP, P K, dS K).  It also finds D, for itself and for the next.
//   * dk, dv: 128 keys stay while 64-row query tiles of all heads of the group stream, so
//     that the sums over a group's heads are sums in tensor memory, in a fixed order and
//     without atomics; four products a tile (S^T, dP^T, dV, dK).  Scores are computed
//     transposed: a thread owns a key.
// Together eight products where five would do: S and dP are computed twice, which costs
// less than adding dQ up over key tiles in memory (64 KB a tile pair), and leaves
// no order to chance; P K makes dQ as exact as D is (below).
//
// Operands.  A product of two operands in shared memory reads 8 KB for each 64 cycles of
// the tensor core, all that shared memory delivers; with the tiles' copies it fell behind by
// a third.  What stays therefore lies in tensor memory, copied there by the compute threads
// from where TMA put it, as P and dS do: a product then reads one operand from shared memory,
// at half its rate, and those of 64 columns run at full rate (33.8 cycles of 32; from shared memory 49).
// Tensor memory has room for all that stays at d = 64, and for one of its two tensors at d = 128.
//
// Measured, four causal samples of 1000 to 8192 tokens (17335), 32 heads on 8, d = 128: dq 1060 us, dk and
// dv 1005 us, the tensor core busy for 70 and 76 % of them; 1.66 PFLOP/s of the eight products,
// near what the power limit leaves. 31 samples of up to 1500 tokens, 16 heads on 2, d = 64, full:
// 230 and 232 us, 39 and 44 % busy; there the threads' part of a tile takes longer than its products.
//
// D from the bf16 o is off by half a bf16 step of it, and by what the rounding of P cost o.  A row's dS
// have that error in common: it moves dq by as much times the row's mean key, which for
// scores that single out a few keys, or keys that lie far to one side, is more than all other roundings
// together.  The dq kernel therefore corrects dq for the difference to D = sum_j P_ij dP_ij (see there).
// Query tiles that see 64 keys or fewer take that sum as D from the start, which their threads have
// in registers before dS is needed: where a query sees its own key alone, dS is zero.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_packed.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

__device__ unsigned int g_packed_bwd_error;
// Set by the first launch: until then the record above is clean and need not be copied, which takes 10 us.
std::atomic<bool> g_packed_bwd_used{false};

constexpr int kDqMma = 3, kDkMma = 3;  // MMA warps
constexpr int kCompute = 256;
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kDqThreads = kCompute + 32 + 32 * kDqMma, kDkThreads = kCompute + 32 + 32 * kDkMma;
constexpr float kLog2e = 1.44269504088896340736f;

struct BwdParams {
  PackedHeader* header;
  const PackedEntry* list;
  const CUtensorMap* maps;  // four a sequence: q, k, v, dO
  const float* lse;
  float* D;
  const __nv_bfloat16* o;
  const __nv_bfloat16* dO;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  long long o_token, o_head, dO_token, dO_head, dq_token, dq_head, dk_token, dk_head, dv_token, dv_head;
  int total_q;
  int P, TT, TT64, heads, per_kv, Hkv, chunk;  // TT64: query tokens in 64 rows, TT: in two such boxes
  float scale, scale_log2;
};

constexpr int kBwdRing = 2;  // items in flight between the roles of a CTA
constexpr int kStages = 5;  // of 64 streamed rows of two tensors
constexpr uint32_t kBarBytes = 512;

// Barriers of both kernels.  The two halves of a stage have barriers of their own in the dq
// kernel, where a key tile is needed longer than a value tile.
struct BwdBars {
  uint64_t res_full, res_empty;  // what stays: copied to shared memory; read from there
  uint64_t a_ready;              // and written to tensor memory
  uint64_t x_full[kStages], x_empty[kStages];
  uint64_t y_full[kStages], y_empty[kStages];
  uint64_t s_full[2], s_done[2];  // scores computed; P written over them
  uint64_t dp_full[2], ds_ready[2];
  uint64_t dp_read[2];
  uint64_t done[2];  // the products that read a buffer's P and dS
  uint64_t dx_ready, de_ready;  // (dq) halves of a row's D from o, and of its exact D
  uint64_t acc_done, acc_free;
  uint64_t item_full[kBwdRing], item_empty[kBwdRing];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  PackedItem item[kBwdRing];
};
static_assert(sizeof(BwdBars) <= kBarBytes, "barrier block overruns its shared memory");

// A wait's loop out of line: the code of the kernels stays small.
__device__ __noinline__ bool wait_loop(uint64_t* bar, uint32_t par, BwdBars* b, uint32_t code) {
  return mbar_wait(bar, par, &b->abort_flag, &g_packed_bwd_error, code);
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t par, BwdBars* b, uint32_t code) {
  return mbar_try_wait(smem_u32(bar), par) || wait_loop(bar, par, b, code);
}
// The same by a whole warp, with one answer.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t par, BwdBars* b, uint32_t code) {
  return __all_sync(0xffffffffu, wait(bar, par, b, code));
}

// Adds `bytes` to the transaction count of the current phase of `bar` without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}

// Barriers and tensor memory; rows of [zero, zero + bytes) that no box fills are zeroed.
// `users`: MMA warps whose products read a stage, and which write an accumulator; `mma`: all;
// `resident`: those that read what stays from shared memory.
// `code`: of the record where shared memory does not lie as the tiles' swizzle needs it.
// Returns false when an earlier CTA recorded a timeout.
__device__ __forceinline__ bool bwd_init(BwdBars* bars, int warp, const uint8_t* smem, uint8_t* zero,
                                         uint32_t bytes, int users, int mma, int resident, uint32_t code) {
  if (threadIdx.x == 0) {
    // the swizzle of tiles counts from 1024-byte boundaries
    if ((smem_u32(smem) & 1023u) != 0) atomicCAS(&g_packed_bwd_error, 0u, kDevTimeoutMask | code);
    mbar_init(&bars->res_full, 1);
    mbar_init(&bars->res_empty, kCompute + resident);
    mbar_init(&bars->a_ready, kCompute);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bars->x_full[s], 1);
      mbar_init(&bars->x_empty[s], users);
      mbar_init(&bars->y_full[s], 1);
      mbar_init(&bars->y_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&bars->s_full[b], 1);
      mbar_init(&bars->s_done[b], kCompute);
      mbar_init(&bars->dp_full[b], 1);
      mbar_init(&bars->dp_read[b], kCompute);
      mbar_init(&bars->done[b], 1);
      mbar_init(&bars->ds_ready[b], kCompute);
    }
    mbar_init(&bars->dx_ready, kCompute);
    mbar_init(&bars->de_ready, kCompute);
    mbar_init(&bars->acc_done, users);
    mbar_init(&bars->acc_free, kCompute);
    for (int r = 0; r < kBwdRing; ++r) {
      mbar_init(&bars->item_full[r], 1);
      mbar_init(&bars->item_empty[r], kCompute / 32 + mma);  // the compute and MMA warps
    }
    mbar_init(&bars->drain, mma);
    bars->abort_flag = (*static_cast<volatile unsigned int*>(&g_packed_bwd_error) != 0) ? 1 : 0;
    fence_mbar_init();
  }
  if (bytes > 0) {
    for (uint32_t i = threadIdx.x; i < bytes / 16; i += blockDim.x)
      reinterpret_cast<uint4*>(zero)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  __syncthreads();
  if (bars->abort_flag) return false;
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  return true;
}

// An item, waited for, and given back once it has been read (by whole warps).
__device__ __forceinline__ bool item_wait(BwdBars* bars, int t, uint32_t code) {
  return warp_wait(&bars->item_full[t % kBwdRing], (t / kBwdRing) & 1, bars, code);
}
__device__ __forceinline__ void item_done(BwdBars* bars, int r) {
  __syncwarp();
  if (lane_id() == 0) mbar_arrive(&bars->item_empty[r]);
}

__device__ __forceinline__ void bwd_teardown(BwdBars* bars, int warp, uint32_t tmem, uint32_t code) {
  if (warp == kMmaWarp) wait(&bars->drain, 0, bars, code);
  if (bars->abort_flag) {
    // let any bulk copy already in flight land before the CTA exits
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// K-major operand descriptor for k-step kk of a [64 rows][D] swizzled tile.
__device__ __forceinline__ uint64_t kmajor_desc(uint32_t base, int kk) {
  return sdesc_sw128(base + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024);
}
// MN-major operand descriptor (the tile's 64 rows are the K dimension) for k-step kk.
__device__ __forceinline__ uint64_t mnmajor_desc(uint32_t base, int kk) {
  return sdesc_sw128(base + kk * 2048, 8192, 1024);
}
// Tensor-memory column of k-step kk (16 score columns) of a bf16 operand packed inside the two
// 32-column halves of a 64-column fp32 region, each in its half's first 16 columns.
__device__ __forceinline__ uint32_t packed_a_col(int kk) {
  return static_cast<uint32_t>((kk >> 1) * 32 + (kk & 1) * 8);
}

__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[32]) {
  tmem_ld32(addr, r);
  tmem_ld_wait();
  reg_pin(r);
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&w)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
      "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]),
      "r"(w[15])
      : "memory");
}

// Half of row tr of a [128 rows][D] swizzled tile in shared memory (zeros unless `valid`), as it
// lies in registers and, packed as a product's A operand, in tensor memory.
template <int D>
__device__ __forceinline__ void load_half_row(const uint8_t* tile, int tr, int half, bool valid,
                                              uint32_t (&w)[D / 4]) {
#pragma unroll
  for (int e = 0; e < D / 16; ++e) {
    const int c = half * (D / 16) + e;  // 16-byte chunk of the row
    uint4 x = make_uint4(0, 0, 0, 0);
    if (valid)
      x = *reinterpret_cast<const uint4*>(tile + (c >> 3) * 16384 + tr * 128 + (((c & 7) ^ (tr & 7)) << 4));
    w[4 * e] = x.x, w[4 * e + 1] = x.y, w[4 * e + 2] = x.z, w[4 * e + 3] = x.w;
  }
}
// Zeros there, for products that read the tile from shared memory.
template <int D>
__device__ __forceinline__ void zero_half_row(uint8_t* tile, int tr, int half) {
#pragma unroll
  for (int e = 0; e < D / 16; ++e) {
    const int c = half * (D / 16) + e;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * 16384 + tr * 128 + (((c & 7) ^ (tr & 7)) << 4)) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
}
template <int D>
__device__ __forceinline__ void store_half_row(uint32_t addr, int half, const uint32_t (&w)[D / 4]) {
  if constexpr (D == 128)
    tmem_st32(addr + 32 * half, w);
  else
    tmem_st16(addr + 16 * half, w);
}

// Stores 32 fp32 accumulator columns of this lane's row times `mul` as bf16, at dst + off
// (off < 0: the row does not exist), the rows of a 4-lane group together.
__device__ __forceinline__ void store_acc32(uint32_t addr, float mul, __nv_bfloat16* dst, long long off) {
  const int lane = threadIdx.x & 31;
  uint32_t r[32], w[16];
  tmem_ld32(addr, r);
  tmem_ld_wait();
  reg_pin(r);
#pragma unroll
  for (int e = 0; e < 16; ++e)
    w[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * mul, __uint_as_float(r[2 * e + 1]) * mul);
  transpose_chunks<4>(w);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long o = __shfl_sync(0xffffffffu, off, (lane & ~3) + k);
    if (o >= 0)
      *reinterpret_cast<uint4*>(dst + o + (lane & 3) * 8) =
          make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
}

// The same of x - d y for two accumulators x and y.
__device__ __forceinline__ void store_acc32(uint32_t x_addr, uint32_t y_addr, float d, float mul, __nv_bfloat16* dst,
                                            long long off) {
  const int lane = threadIdx.x & 31;
  uint32_t x[32], y[32], w[16];
  tmem_ld32(x_addr, x);
  tmem_ld32(y_addr, y);
  tmem_ld_wait();
  reg_pin(x);
  reg_pin(y);
#pragma unroll
  for (int e = 0; e < 32; ++e)
    x[e] = __float_as_uint(mul * fmaf(-d, __uint_as_float(y[e]), __uint_as_float(x[e])));
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
  transpose_chunks<4>(w);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const long long o = __shfl_sync(0xffffffffu, off, (lane & ~3) + k);
    if (o >= 0)
      *reinterpret_cast<uint4*>(dst + o + (lane & 3) * 8) =
          make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
}

__device__ __forceinline__ void store_zeros(__nv_bfloat16* dst, int n) {
  for (int e = 0; e < n / 8; ++e) reinterpret_cast<uint4*>(dst)[e] = make_uint4(0u, 0u, 0u, 0u);
}

// Tensor memory of both kernels: scores of 64 streamed rows, dP, two accumulators, and what stays.  P and dS lie
// over the scores, whose bits they take half of: so dP is free again once it has been read, and its next
// product does not wait for those of P and dS.  At d = 64 there are two buffers of scores and of dP (step
// g's in buffer g & 1).  At d = 128 there is room for two of scores or for both tensors that stay, by DP_SMEM,
// the operands that dP's product reads from shared memory: 1, scores in one buffer; 2, one tensor stays in
// shared memory until the item's last dP, and its product runs at the speed of shared memory (49 cycles where
// 33 would do).
template <int D, int DP_SMEM>
struct BwdTmem {
  static constexpr bool kBothStay = DP_SMEM == 1;
  static constexpr int kSBufs = D == 128 && kBothStay ? 1 : 2, kDpBufs = D == 64 ? 2 : 1;
  static constexpr uint32_t kDp = 64 * kSBufs;
  static constexpr uint32_t kAcc0 = kDp + 64 * kDpBufs, kAcc1 = kAcc0 + D;
  static constexpr uint32_t kStay0 = kAcc1 + D;  // Q or K, the scores' operand
  __host__ __device__ static constexpr uint32_t stay1_col() { return kStay0 + D / 2; }  // dO or V, dP's
  // a step's buffers, and the parities of their barriers
  __host__ __device__ static constexpr int s_buf(int step) { return kSBufs == 2 ? step & 1 : 0; }
  __host__ __device__ static constexpr uint32_t s_par(int step) { return kSBufs == 2 ? (step >> 1) & 1 : step & 1; }
  __host__ __device__ static constexpr uint32_t s_col(int step) { return 64u * s_buf(step); }
  __host__ __device__ static constexpr int dp_buf(int step) { return kDpBufs == 2 ? step & 1 : 0; }
  __host__ __device__ static constexpr uint32_t dp_par(int step) { return kDpBufs == 2 ? (step >> 1) & 1 : step & 1; }
  __host__ __device__ static constexpr uint32_t dp_col(int step) { return kDp + 64u * dp_buf(step); }
};
static_assert(BwdTmem<64, 1>::stay1_col() + 32 <= 512 && BwdTmem<128, 1>::stay1_col() + 64 <= 512 &&
                  BwdTmem<128, 2>::kStay0 + 64 <= 512,
              "512 columns");

// ============================================================ dQ
// D is needed before the loop over key tiles has seen the whole row.  The loop therefore takes D' = sum_c
// dO o from the bf16 o, and beside dQ' = sum_j P_ij (dP_ij - D') k_j it finds D = sum_j P_ij dP_ij in fp32 and
// R = sum_j P_ij k_j, one more product; dQ = scale (dQ' - (D - D') R) is then free of the error that o's and P's
// rounding put into D', and D goes to the dk, dv kernel.
template <int D, int DP_SMEM>
struct DqLayout : BwdTmem<D, DP_SMEM> {
  static constexpr int kChunks = D / 64;
  static constexpr uint32_t kRes = 128u * D * 2, kTile = 64u * D * 2;
  static constexpr uint32_t kQ = 0, kDO = kRes, kK = 2 * kRes, kV = kK + kStages * kTile;
  static constexpr uint32_t kDx = kV + kStages * kTile;  // [D' | D][half][128]
  static constexpr uint32_t kBar = kDx + 2048;
  static constexpr uint32_t kUsed = kBar + kBarBytes;
  static constexpr uint32_t kSmem = kUsed > 118784u ? kUsed : 118784u;  // one CTA an SM
};
static_assert(DqLayout<128, 1>::kSmem <= 232448, "227 KB a CTA");

// Key tiles of an item.
__device__ __forceinline__ int dq_tiles(const PackedItem& it, int TT, bool causal) {
  return (packed_keys(min((it.e.tile + 1) * TT, it.e.n) - 1, it.e.n, it.e.m, causal) + 63) >> 6;
}

template <int D, bool CAUSAL, int DP_SMEM>
__global__ void __launch_bounds__(kDqThreads, 1) fa_packed_dq_kernel(const __grid_constant__ BwdParams p) {
  using L = DqLayout<D, DP_SMEM>;
  extern __shared__ __align__(1024) uint8_t smem[];
  BwdBars* bars = reinterpret_cast<BwdBars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!bwd_init(bars, warp, smem, smem, 0, 1, kDqMma, L::kBothStay ? 0 : 1, 0x23ff)) return;
  const uint32_t tmem = bars->tmem_base;
  grid_dependency_wait();
  grid_dependency_launch();

  if (warp == kTmaWarp) {
    const uint32_t q_bytes = static_cast<uint32_t>(p.P * p.TT64) * 128u * L::kChunks;
    int kvb = 0, tl = 0;  // key tiles and items with loads so far
    auto claim = [&]() {
      PackedItem x;
      x.head = -1;
      if (lane == 0) x = packed_claim(p.header, p.list, 0, p.heads, p.chunk);
      return x;
    };
    PackedItem it = claim();
    for (int t = 0;; ++t) {
      const int r = t % kBwdRing;
      if (!warp_wait(&bars->item_empty[r], ((t / kBwdRing) & 1) ^ 1, bars, 0x2104)) break;
      if (lane == 0) {
        bars->item[r] = it;
        mbar_arrive(&bars->item_full[r]);
      }
      __syncwarp();
      it = bars->item[r];
      __syncwarp();
      if (it.head < 0) break;
      const int n = dq_tiles(it, p.TT, CAUSAL);
      if (n == 0) {
        it = claim();
        continue;
      }
      if (tl > 0 && !warp_wait(&bars->res_empty, (tl - 1) & 1, bars, 0x2103)) break;
      bool ok = true;
      PackedItem next = it;
      if (lane == 0) {
        const CUtensorMap* maps = p.maps + 4ll * it.e.seq;
#pragma unroll
        for (int i = 0; i < 4; ++i) tensormap_acquire(maps + i);
        const int kh = it.head / p.per_kv;
        mbar_arrive_expect_tx(&bars->res_full, 4 * q_bytes);
#pragma unroll
        for (int c = 0; c < 2 * L::kChunks; ++c) {  // two boxes of 64 rows a column
          const int col = c >> 1, half = c & 1, tok = it.e.tile * p.TT + half * p.TT64;
          const uint32_t at = col * 16384 + half * 8192;
          tma_load_4d(smem + L::kQ + at, maps, &bars->res_full, col * 64, 0, tok, it.head);
          tma_load_4d(smem + L::kDO + at, maps + 3, &bars->res_full, col * 64, 0, tok, it.head);
        }
        auto load = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, int j) {
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c) tma_load_3d(dst + c * 8192, map, bar, c * 64, j * 64, kh);
        };
        for (int j = 0; j < n; ++j) {
          const int s = (kvb + j) % kStages;
          const uint32_t par = (((kvb + j) / kStages) & 1) ^ 1;
          if (!(ok = wait(&bars->x_empty[s], par, bars, 0x2101))) break;
          mbar_arrive_expect_tx(&bars->x_full[s], L::kTile);
          load(smem + L::kK + s * L::kTile, maps + 1, &bars->x_full[s], j);
          if (!(ok = wait(&bars->y_empty[s], par, bars, 0x2102))) break;
          mbar_arrive_expect_tx(&bars->y_full[s], L::kTile);
          load(smem + L::kV + s * L::kTile, maps + 2, &bars->y_full[s], j);
          // the next item is asked for while the last tiles are under way
          if (j == max(n - 2, 0)) next = packed_claim(p.header, p.list, 0, p.heads, p.chunk);
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      kvb += n;
      ++tl;
      it = next;
    }
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // Three warps issue, S, dP, and P K and dS K: 8 products take 210 cycles to issue in a kernel that does
    // nothing else and up to 500 in one like this, a wait that is over 70; where one warp issued dP and dQ
    // it took 1350 cycles a step.  The whole warp runs the loop on values that are the same in all
    // lanes, so that descriptors lie in uniform registers, where the instruction wants them;
    // one elected lane issues.
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, D, false, true);
    const int role = warp - kMmaWarp;
    const uint32_t tm = uniform(tmem), sK = uniform(smem_u32(smem + L::kK)), sV = uniform(smem_u32(smem + L::kV));
    [[maybe_unused]] const uint32_t sdO = uniform(smem_u32(smem + L::kDO));
    int kvb = 0, tl = 0;
    for (int t = 0;; ++t) {
      if (!item_wait(bars, t, 0x221b)) break;
      const PackedItem it = bars->item[t % kBwdRing];
      item_done(bars, t % kBwdRing);
      if (uniform(it.head) < 0) break;
      const int n = uniform(dq_tiles(it, p.TT, CAUSAL));
      if (n == 0) continue;
      if (!warp_wait(&bars->a_ready, tl & 1, bars, 0x2210)) break;
      bool ok = true;
      if (role == 0) {
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int pos = kvb + j, s = pos % kStages, before = pos - L::kSBufs;
          // (the P and dS in the buffer have been multiplied)
          if (!(ok = warp_wait(&bars->x_full[s], (pos / kStages) & 1, bars, 0x2211) &&
                     (before < 0 || warp_wait(&bars->done[L::s_buf(before)], L::s_par(before), bars, 0x2212))))
            break;
          tc_fence_after_sync();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ts(tm + L::s_col(pos), tm + L::kStay0 + kk * 8, kmajor_desc(sK + s * L::kTile, kk), idesc_s,
                      kk > 0 ? 1u : 0u);
            umma_commit(&bars->s_full[L::s_buf(pos)]);
          }
          __syncwarp();
        }
      } else if (role == 1) {
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int pos = kvb + j, s = pos % kStages, before = pos - L::kDpBufs;
          // (the buffer's last dP has been read)
          if (!(ok = warp_wait(&bars->y_full[s], (pos / kStages) & 1, bars, 0x2213) &&
                     (before < 0 || warp_wait(&bars->dp_read[L::dp_buf(before)], L::dp_par(before), bars, 0x2215))))
            break;
          tc_fence_after_sync();
          if (elect_one()) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              if constexpr (L::kBothStay)
                umma_ts(tm + L::dp_col(pos), tm + L::stay1_col() + kk * 8, kmajor_desc(sV + s * L::kTile, kk), idesc_s,
                        kk > 0 ? 1u : 0u);
              else
                umma_ss(tm + L::dp_col(pos), sdesc_sw128(sdO + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                        kmajor_desc(sV + s * L::kTile, kk), idesc_s, kk > 0 ? 1u : 0u);
            }
            umma_commit(&bars->dp_full[L::dp_buf(pos)]);
            umma_commit(&bars->y_empty[s]);
            if (!L::kBothStay && j + 1 == n) umma_commit(&bars->res_empty);
          }
          __syncwarp();
        }
      } else {
        // R += P K_j and dQ' += dS K_j (A = bf16 in tensor memory over the scores)
        auto issue_acc = [&](uint32_t acc, uint32_t a, int s, bool first) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ts(acc, a + packed_a_col(kk), mnmajor_desc(sK + s * L::kTile, kk), idesc_acc,
                    (!first || kk > 0) ? 1u : 0u);
        };
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int pos = kvb + j, s = pos % kStages;
          // an item's first overwrite the accumulators that the epilogue before it reads
          if (!(ok = (j > 0 || tl == 0 || warp_wait(&bars->acc_free, (tl - 1) & 1, bars, 0x2216)) &&
                     warp_wait(&bars->s_done[L::s_buf(pos)], L::s_par(pos), bars, 0x2217)))
            break;
          tc_fence_after_sync();
          if (elect_one()) issue_acc(tm + L::kAcc0, tm + L::s_col(pos), s, j == 0);
          __syncwarp();
          if (!(ok = warp_wait(&bars->ds_ready[L::s_buf(pos)], L::s_par(pos), bars, 0x2214))) break;
          tc_fence_after_sync();
          if (elect_one()) {
            issue_acc(tm + L::kAcc1, tm + L::s_col(pos) + 16, s, j == 0);
            umma_commit(&bars->done[L::s_buf(pos)]);
            umma_commit(&bars->x_empty[s]);
            if (j + 1 == n) umma_commit(&bars->acc_done);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      kvb += n;
      ++tl;
    }
    __syncwarp();
    if (elect_one()) umma_commit(&bars->drain);
    __syncwarp();
  } else {
    const int g = threadIdx.x >> 7;    // half of the score columns
    const int tr = threadIdx.x & 127;  // row within the tile, TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm = tmem + lane_off;
    const int box = tr >> 6, box_tok = (tr & 63) / p.P, row_head = (tr & 63) - box_tok * p.P;
    const bool row_in = box_tok < p.TT64;
    const int row_tok = box * p.TT64 + box_tok;
    // (an item's parts of D' have been read by all threads before any writes the next's: it has waited
    // for the item's dQ, which needs the last dS of all; and its parts of D before any writes the
    // next's, since all read them before they give that item's parts of D')
    float* dx = reinterpret_cast<float*>(smem + L::kDx);
    float* de = dx + 256;
    int nb = 0, tl = 0, te = 0;  // steps, items with products, and of those with D in parts so far
    // dQ of the item before: stored when the next one's Q and dO lie in tensor memory, so that its
    // first products run meanwhile
    bool pending = false, in_parts = false;
    long long pending_at = -1, pending_vec = -1;
    float D0 = 0.0f;  // its D'
    auto epilogue = [&]() {
      if (!pending) return true;
      float Di = D0;
      if (in_parts) {
        if (!warp_wait(&bars->de_ready, te++ & 1, bars, 0x2316)) return false;
        Di = de[tr] + de[128 + tr];
      }
      if (g == 0 && pending_at >= 0) p.D[pending_vec] = Di;
      if (!warp_wait(&bars->acc_done, (tl - 1) & 1, bars, 0x2312)) return false;
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        store_acc32(tm + L::kAcc1 + (D / 2) * g + c * 32, tm + L::kAcc0 + (D / 2) * g + c * 32, Di - D0, p.scale,
                    p.dq + c * 32, pending_at);
      // the accumulators have been read: the next item may overwrite them
      tc_fence_before_sync();
      mbar_arrive(&bars->acc_free);
      pending = false;
      return true;
    };
    for (int ti = 0;; ++ti) {
      if (!item_wait(bars, ti, 0x2304)) break;
      const PackedItem it = bars->item[ti % kBwdRing];
      item_done(bars, ti % kBwdRing);
      if (it.head < 0) {
        epilogue();
        break;
      }
      const int n = dq_tiles(it, p.TT, CAUSAL);
      const int tok0 = it.e.tile * p.TT, tok = tok0 + row_tok;
      const bool valid = row_in && tok < it.e.n;
      const int head = it.head * p.P + row_head, m = it.e.m, off = m - it.e.n;
      const long long token = it.e.q0 + tok;
      const long long vec = static_cast<long long>(head) * p.total_q + token;
      if (n == 0) {  // no key is seen
        if (valid) {
          store_zeros(p.dq + token * p.dq_token + head * p.dq_head + (D / 2) * g, D / 2);
          if (g == 0) p.D[vec] = 0.0f;
        }
        continue;
      }
      // asked for here, used below
      float lse = valid ? p.lse[vec] : INFINITY;
      uint4 o_row[D / 16];
      if (n > 1 && valid) {
        const uint4* a = reinterpret_cast<const uint4*>(p.o + token * p.o_token + head * p.o_head + (D / 2) * g);
#pragma unroll
        for (int e = 0; e < D / 16; ++e) o_row[e] = a[e];
      }
      bool ok = true;
      float Di = 0.0f;
      // the halves' parts of D' (of D itself in an item of one step) meet in shared memory
      auto join = [&](float part) {
        dx[g * 128 + tr] = part;
        mbar_arrive(&bars->dx_ready);
        ok = warp_wait(&bars->dx_ready, tl & 1, bars, 0x2313);
        Di = dx[tr] + dx[128 + tr];
      };
      // Q and dO to tensor memory: the products of the item before that read them are done (its
      // last scores and dP have been waited for)
      if (!warp_wait(&bars->res_full, tl & 1, bars, 0x2315)) break;
      float part = 0.0f;
      {
        uint32_t w[D / 4];
        load_half_row<D>(smem + L::kQ, tr, g, valid, w);
        store_half_row<D>(tm + L::kStay0, g, w);
        // (a row that sees no key counts as one of zeros, whatever its dO holds)
        const bool live = valid && (!CAUSAL || tok + off >= 0);
        load_half_row<D>(smem + L::kDO, tr, g, live, w);
        if constexpr (L::kBothStay)
          store_half_row<D>(tm + L::stay1_col(), g, w);
        else if (valid && !live)
          zero_half_row<D>(smem + L::kDO, tr, g);
        mbar_arrive(&bars->res_empty);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars->a_ready);
        if (n > 1 && valid) {
#pragma unroll
          for (int e = 0; e < D / 16; ++e) {
            const uint32_t xs[4] = {o_row[e].x, o_row[e].y, o_row[e].z, o_row[e].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              part = fmaf(__uint_as_float(xs[i] << 16), __uint_as_float(w[4 * e + i] << 16), part);
              part = fmaf(__uint_as_float(xs[i] & 0xffff0000u), __uint_as_float(w[4 * e + i] & 0xffff0000u), part);
            }
          }
        }
      }
      if (!epilogue()) break;
      if (n > 1) {
        join(part);
        if (!ok) break;
      }
      // a row behind the sequence: P = 2^-inf; one that sees no key: all of it is masked; one that sees keys whose
      // scores are all -inf: lse = -inf, P = 2^(-inf + inf), NaN by the definition
      asm volatile("" : "+f"(lse));  // (not multiplied where it was asked for, which would wait for it there)
      const float lse2 = lse * kLog2e;
      const uint32_t col0 = 32u * g;
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nl2 = make_float2(-lse2, -lse2);
      float2 exact = make_float2(0.f, 0.f);  // sum of P dP
      for (int j = 0; j < n; ++j) {
        const int step = nb + j;
        if (!(ok = warp_wait(&bars->s_full[L::s_buf(step)], L::s_par(step), bars, 0x2311))) break;
        tc_fence_after_sync();
        uint32_t pr[32];
        tmem_ld(tm + L::s_col(step) + col0, pr);
        const int kv0 = j * 64;
        const bool need_mask = (CAUSAL && kv0 + 63 > tok0 + off) || kv0 + 64 > m;
        auto exp_cols = [&](auto masked, int lim) {
#pragma unroll
          for (int c = 0; c < 32; c += 2) {
            const float2 x =
                __ffma2_rn(make_float2(__uint_as_float(pr[c]), __uint_as_float(pr[c + 1])), sc2, nl2);
            float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
            if (masked) {
              if (c > lim) p0 = 0.0f;
              if (c + 1 > lim) p1 = 0.0f;
            }
            pr[c] = __float_as_uint(p0);
            pr[c + 1] = __float_as_uint(p1);
          }
        };
        if (need_mask)
          exp_cols(std::true_type{}, (CAUSAL ? min(tok + off, m - 1) : m - 1) - kv0 - static_cast<int>(col0));
        else
          exp_cols(std::false_type{}, 0);
        {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c)
            pk[c] = pack_bf16x2(__uint_as_float(pr[2 * c]), __uint_as_float(pr[2 * c + 1]));
          tmem_st16(tm + L::s_col(step) + col0, pk);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars->s_done[L::s_buf(step)]);
        if (!(ok = warp_wait(&bars->dp_full[L::dp_buf(step)], L::dp_par(step), bars, 0x2314))) break;
        tc_fence_after_sync();
        uint32_t rr[32];
        tmem_ld(tm + L::dp_col(step) + col0, rr);
        tc_fence_before_sync();
        mbar_arrive(&bars->dp_read[L::dp_buf(step)]);
        auto add_exact = [&]() {
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            exact = __ffma2_rn(make_float2(__uint_as_float(pr[e]), __uint_as_float(pr[e + 1])),
                               make_float2(__uint_as_float(rr[e]), __uint_as_float(rr[e + 1])), exact);
        };
        if (D == 64 || n == 1) add_exact();
        if (n == 1) {
          join(exact.x + exact.y);
          if (!ok) break;
        }
        const float2 nD2 = make_float2(-Di, -Di);
        uint32_t ds[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 x = __fmul2_rn(
              make_float2(__uint_as_float(pr[2 * e]), __uint_as_float(pr[2 * e + 1])),
              __fadd2_rn(make_float2(__uint_as_float(rr[2 * e]), __uint_as_float(rr[2 * e + 1])), nD2));
          ds[e] = pack_bf16x2(x.x, x.y);
        }
        tmem_st16(tm + L::s_col(step) + col0 + 16, ds);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars->ds_ready[L::s_buf(step)]);
        // (at d = 128 while the products run, 1.6 % faster there; at d = 64, where the threads bound the
        // kernel, 31 full samples of up to 1500 tokens take 254 us that way, and 234 the other)
        if (D == 128 && n > 1) add_exact();
      }
      if (!ok) break;
      if (n > 1) {
        de[g * 128 + tr] = exact.x + exact.y;
        mbar_arrive(&bars->de_ready);
      }
      pending = true;
      in_parts = n > 1;
      D0 = Di;
      pending_vec = vec;
      pending_at = valid ? token * p.dq_token + head * p.dq_head + (D / 2) * g : -1;
      nb += n;
      ++tl;
    }
  }
  bwd_teardown(bars, warp, tmem, 0x22ff);
}

// ============================================================ dK / dV
template <int D, int DP_SMEM>
struct DkLayout : BwdTmem<D, DP_SMEM> {
  static constexpr int kChunks = D / 64;
  static constexpr uint32_t kRes = 128u * D * 2, kTile = 64u * D * 2;
  static constexpr uint32_t kK = 0, kV = kRes, kQ = 2 * kRes, kDO = kQ + kStages * kTile;
  static constexpr uint32_t kVec = kDO + kStages * kTile;  // [stage][-lse2 | -D][64]
  static constexpr uint32_t kBar = kVec + kStages * 512;
  static constexpr uint32_t kUsed = kBar + kBarBytes;
  static constexpr uint32_t kSmem = kUsed > 118784u ? kUsed : 118784u;  // one CTA an SM
};
static_assert(DkLayout<128, 1>::kSmem <= 232448, "227 KB a CTA");

// Query tiles (of 64 rows, TT tokens) of a head group that see the item's `keys` keys: the first, and
// how many.
__device__ __forceinline__ int dk_first(const PackedItem& it, int keys, int TT, bool causal) {
  return causal ? max(it.e.tile * keys - (it.e.m - it.e.n), 0) / TT : 0;
}
__device__ __forceinline__ int dk_tiles(const PackedItem& it, int keys, int TT, bool causal) {
  return max((it.e.n + TT - 1) / TT - dk_first(it, keys, TT, causal), 0);
}

template <int D, bool CAUSAL, int DP_SMEM>
__global__ void __launch_bounds__(kDkThreads, 1) fa_packed_dkdv_kernel(const __grid_constant__ BwdParams p) {
  using L = DkLayout<D, DP_SMEM>;
  extern __shared__ __align__(1024) uint8_t smem[];
  BwdBars* bars = reinterpret_cast<BwdBars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int TT = p.TT64;
  if (!bwd_init(bars, warp, smem, smem + L::kQ, p.P * TT < 64 ? 2 * kStages * L::kTile : 0, 1, kDkMma,
                    L::kBothStay ? 0 : 1, 0x33ff))
    return;
  const uint32_t tmem = bars->tmem_base;
  grid_dependency_wait();

  if (warp == kTmaWarp) {
    const uint32_t q_bytes = static_cast<uint32_t>(p.P * TT) * 128u * L::kChunks;
    int row_tok[2], row_head[2];  // of rows lane and lane + 32
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      row_tok[e] = (lane + 32 * e) / p.P;
      row_head[e] = lane + 32 * e - row_tok[e] * p.P;
    }
    int sb = 0, tl = 0;
    auto claim = [&]() {
      PackedItem x;
      x.head = -1;
      if (lane == 0) x = packed_claim(p.header, p.list, 1, p.Hkv, p.chunk);
      return x;
    };
    PackedItem it = claim();
    for (int t = 0;; ++t) {
      const int r = t % kBwdRing;
      if (!warp_wait(&bars->item_empty[r], ((t / kBwdRing) & 1) ^ 1, bars, 0x3104)) break;
      if (lane == 0) {
        bars->item[r] = it;
        mbar_arrive(&bars->item_full[r]);
      }
      __syncwarp();
      it = bars->item[r];
      __syncwarp();
      if (it.head < 0) break;
      const int first = dk_first(it, 128, TT, CAUSAL), per = dk_tiles(it, 128, TT, CAUSAL);
      const int n = per * p.per_kv;
      if (n == 0) {
        it = claim();
        continue;
      }
      const CUtensorMap* maps = p.maps + 4ll * it.e.seq;
      if (tl > 0 && !warp_wait(&bars->res_empty, (tl - 1) & 1, bars, 0x3102)) break;
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) tensormap_acquire(maps + i);
        mbar_arrive_expect_tx(&bars->res_full, 2 * L::kRes);
#pragma unroll
        for (int c = 0; c < 2 * L::kChunks; ++c) {  // two boxes of 64 keys a column
          const int col = c >> 1, half = c & 1, key = it.e.tile * 128 + half * 64;
          tma_load_3d(smem + L::kK + col * 16384 + half * 8192, maps + 1, &bars->res_full, col * 64, key, it.head);
          tma_load_3d(smem + L::kV + col * 16384 + half * 8192, maps + 2, &bars->res_full, col * 64, key, it.head);
        }
      }
      __syncwarp();
      PackedItem next = it;
      bool ok = true;
      int sub = 0, tile = first;
      // lse and D of this lane's rows of a tile, asked for a tile ahead of their use; rows that do
      // not exist, or see nothing: P = 2^-inf
      float lse[2], Dv[2];
      auto ask = [&](int tile, int sub) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = tile * TT + row_tok[e], group = it.head * p.per_kv + sub;
          lse[e] = INFINITY, Dv[e] = 0.0f;
          if (row_tok[e] < TT && tok < it.e.n && (!CAUSAL || tok + it.e.m >= it.e.n)) {
            const long long at = static_cast<long long>(group * p.P + row_head[e]) * p.total_q + it.e.q0 + tok;
            lse[e] = p.lse[at];
            Dv[e] = p.D[at];
          }
        }
      };
      ask(tile, sub);
      for (int j = 0; j < n; ++j) {
        const int s = (sb + j) % kStages, group = it.head * p.per_kv + sub;
        if (!(ok = warp_wait(&bars->x_empty[s], (((sb + j) / kStages) & 1) ^ 1, bars, 0x3101))) break;
        if (lane == 0) {
          mbar_expect_tx(&bars->x_full[s], 2 * q_bytes);
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c) {
            uint8_t* q = smem + L::kQ + s * L::kTile + c * 8192;
            uint8_t* o = smem + L::kDO + s * L::kTile + c * 8192;
            tma_load_4d(q, maps, &bars->x_full[s], c * 64, 0, tile * TT, group);
            tma_load_4d(o, maps + 3, &bars->x_full[s], c * 64, 0, tile * TT, group);
          }
        }
        float* vec = reinterpret_cast<float*>(smem + L::kVec) + s * 128;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          vec[lane + 32 * e] = -lse[e] * kLog2e;
          vec[64 + lane + 32 * e] = -Dv[e];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->x_full[s]);  // (the stage's one arrival)
        if (++tile == first + per) {
          tile = first;
          ++sub;
        }
        if (j + 1 < n) ask(tile, sub);
        if (lane == 0 && j == max(n - 2, 0)) next = packed_claim(p.header, p.list, 1, p.Hkv, p.chunk);
      }
      if (!ok) break;
      sb += n;
      ++tl;
      it = next;
    }
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // Three warps issue (as in the dq kernel): S^T = K Q^T; dP^T = V dO^T; dV += P^T dO and dK += dS^T Q.
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 64, false, false);
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, D, false, true);
    const int role = warp - kMmaWarp;
    const uint32_t tm = uniform(tmem), sV = uniform(smem_u32(smem + L::kV));
    const uint32_t sQ = uniform(smem_u32(smem + L::kQ)), sdO = uniform(smem_u32(smem + L::kDO));
    auto stage_in = [&](int pos) {
      return warp_wait(&bars->x_full[pos % kStages], (pos / kStages) & 1, bars, 0x3205);
    };
    auto issue_dp = [&](int pos, bool last) {
      const uint32_t o = sdO + pos % kStages * L::kTile;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        if constexpr (L::kBothStay)
          umma_ts(tm + L::dp_col(pos), tm + L::stay1_col() + kk * 8, kmajor_desc(o, kk), idesc_s, kk > 0 ? 1u : 0u);
        else
          umma_ss(tm + L::dp_col(pos), sdesc_sw128(sV + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                  kmajor_desc(o, kk), idesc_s, kk > 0 ? 1u : 0u);
      }
      umma_commit(&bars->dp_full[L::dp_buf(pos)]);
      if (!L::kBothStay && last) umma_commit(&bars->res_empty);
    };
    // acc (+)= A x the rows at `tile` (A = bf16 in tensor memory at `a`)
    auto issue_acc = [&](uint32_t acc, uint32_t a, uint32_t tile, bool first) {
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
        umma_ts(acc, a + packed_a_col(kk), mnmajor_desc(tile, kk), idesc_acc, (!first || kk > 0) ? 1u : 0u);
    };
    int sb = 0, tl = 0;
    for (int t = 0;; ++t) {
      if (!item_wait(bars, t, 0x3207)) break;
      const PackedItem it = bars->item[t % kBwdRing];
      item_done(bars, t % kBwdRing);
      if (uniform(it.head) < 0) break;
      const int n = uniform(dk_tiles(it, 128, TT, CAUSAL)) * p.per_kv;
      if (n == 0) continue;
      if (!warp_wait(&bars->a_ready, tl & 1, bars, 0x3201)) break;
      bool ok = true;
      if (role == 0) {
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int pos = sb + j, before = pos - L::kSBufs;
          // (the P and dS in the buffer have been multiplied)
          if (!(ok = stage_in(pos) &&
                     (before < 0 || warp_wait(&bars->done[L::s_buf(before)], L::s_par(before), bars, 0x3202))))
            break;
          tc_fence_after_sync();
          if (elect_one()) {
            const uint32_t q = sQ + pos % kStages * L::kTile;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ts(tm + L::s_col(pos), tm + L::kStay0 + kk * 8, kmajor_desc(q, kk), idesc_s, kk > 0 ? 1u : 0u);
            umma_commit(&bars->s_full[L::s_buf(pos)]);
          }
          __syncwarp();
        }
      } else if (role == 1) {
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int pos = sb + j, before = pos - L::kDpBufs;
          // (the buffer's last dP has been read)
          if (!(ok = stage_in(pos) &&
                     (before < 0 || warp_wait(&bars->dp_read[L::dp_buf(before)], L::dp_par(before), bars, 0x3208))))
            break;
          tc_fence_after_sync();
          if (elect_one()) issue_dp(pos, j + 1 == n);
          __syncwarp();
        }
      } else {
#pragma unroll 1
        for (int j = 0; j < n; ++j) {
          const int pos = sb + j;
          const uint32_t stage = pos % kStages * L::kTile;
          // an item's first overwrites the accumulators that the epilogue before it reads
          if (!(ok = (j > 0 || tl == 0 || warp_wait(&bars->acc_free, (tl - 1) & 1, bars, 0x3206)) &&
                     warp_wait(&bars->s_done[L::s_buf(pos)], L::s_par(pos), bars, 0x3203)))
            break;
          tc_fence_after_sync();
          if (elect_one()) issue_acc(tm + L::kAcc0, tm + L::s_col(pos), sdO + stage, j == 0);
          __syncwarp();
          if (!(ok = warp_wait(&bars->ds_ready[L::s_buf(pos)], L::s_par(pos), bars, 0x3204))) break;
          tc_fence_after_sync();
          if (elect_one()) {
            issue_acc(tm + L::kAcc1, tm + L::s_col(pos) + 16, sQ + stage, j == 0);
            umma_commit(&bars->done[L::s_buf(pos)]);
            umma_commit(&bars->x_empty[pos % kStages]);
            if (j + 1 == n) umma_commit(&bars->acc_done);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      sb += n;
      ++tl;
    }
    __syncwarp();
    if (elect_one()) umma_commit(&bars->drain);
    __syncwarp();
  } else {
    const int g = threadIdx.x >> 7;    // half of the query columns
    const int tr = threadIdx.x & 127;  // key within the tile, TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm = tmem + lane_off;
    const uint32_t col0 = 32u * g;
    int nb = 0, tl = 0;
    // dV and dK of the item before: stored when the next one's K and V lie in tensor memory
    bool pending = false;
    long long pending_k = -1, pending_v = -1;
    auto epilogue = [&]() {
      if (!pending) return true;
      if (!warp_wait(&bars->acc_done, (tl - 1) & 1, bars, 0x3302)) return false;
      tc_fence_after_sync();
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        store_acc32(tm + L::kAcc0 + (D / 2) * g + c * 32, 1.0f, p.dv + c * 32, pending_v);
        store_acc32(tm + L::kAcc1 + (D / 2) * g + c * 32, p.scale, p.dk + c * 32, pending_k);
      }
      // the accumulators have been read: the next item may overwrite them
      tc_fence_before_sync();
      mbar_arrive(&bars->acc_free);
      pending = false;
      return true;
    };
    for (int ti = 0;; ++ti) {
      if (!item_wait(bars, ti, 0x3305)) break;
      const PackedItem it = bars->item[ti % kBwdRing];
      item_done(bars, ti % kBwdRing);
      if (it.head < 0) {
        epilogue();
        break;
      }
      const int first = dk_first(it, 128, TT, CAUSAL), per = dk_tiles(it, 128, TT, CAUSAL);
      const int n = per * p.per_kv;
      const int key0 = it.e.tile * 128, key = key0 + tr;
      const bool valid = key < it.e.m;
      const long long token = it.e.k0 + key;
      const long long at_k = valid ? token * p.dk_token + it.head * p.dk_head + (D / 2) * g : -1;
      const long long at_v = valid ? token * p.dv_token + it.head * p.dv_head + (D / 2) * g : -1;
      if (n == 0) {  // no query sees the tile
        if (valid) {
          store_zeros(p.dk + at_k, D / 2);
          store_zeros(p.dv + at_v, D / 2);
        }
        continue;
      }
      // K (and V) to tensor memory: the products of the item before that read them are done (its last
      // scores and dP have been waited for)
      if (!warp_wait(&bars->res_full, tl & 1, bars, 0x3307)) break;
      {
        uint32_t w[D / 4];
        load_half_row<D>(smem + L::kK, tr, g, true, w);
        store_half_row<D>(tm + L::kStay0, g, w);
        if constexpr (L::kBothStay) {
          load_half_row<D>(smem + L::kV, tr, g, true, w);
          store_half_row<D>(tm + L::stay1_col(), g, w);
        }
      }
      mbar_arrive(&bars->res_empty);
      tmem_st_wait();
      tc_fence_before_sync();
      mbar_arrive(&bars->a_ready);
      if (!epilogue()) break;
      bool ok = true;
      int tile = first;
      // causal: query token i sees the key where i >= key - (m - n)
      const int from = key - (it.e.m - it.e.n);
      const int last_from = key0 + 127 - (it.e.m - it.e.n);
      const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
      for (int j = 0; j < n; ++j) {
        const int step = nb + j;
        const float* nlse = reinterpret_cast<const float*>(smem + L::kVec) + (step % kStages) * 128;
        if (!(ok = warp_wait(&bars->s_full[L::s_buf(step)], L::s_par(step), bars, 0x3301))) break;
        tc_fence_after_sync();
        uint32_t pr[32];
        tmem_ld(tm + L::s_col(step) + col0, pr);
        const float4* lse4 = reinterpret_cast<const float4*>(nlse + col0);
        auto exp_cols = [&](auto masked, int lim) {
#pragma unroll
          for (int c4 = 0; c4 < 8; ++c4) {
            const float4 l4 = lse4[c4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int c = 4 * c4 + 2 * h;
              const float2 x =
                  __ffma2_rn(make_float2(__uint_as_float(pr[c]), __uint_as_float(pr[c + 1])), sc2,
                             h ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y));
              float p0 = ex2_approx(x.x), p1 = ex2_approx(x.y);
              if (masked) {  // queries before the key
                if (c < lim) p0 = 0.0f;
                if (c + 1 < lim) p1 = 0.0f;
              }
              pr[c] = __float_as_uint(p0);
              pr[c + 1] = __float_as_uint(p1);
            }
          }
        };
        // row r of the tile is token tile * TT + r / P
        if (CAUSAL && tile * TT < last_from)
          exp_cols(std::true_type{}, min(max(from - tile * TT, 0), 64) * p.P - static_cast<int>(col0));
        else
          exp_cols(std::false_type{}, 0);
        {
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c)
            pk[c] = pack_bf16x2(__uint_as_float(pr[2 * c]), __uint_as_float(pr[2 * c + 1]));
          tmem_st16(tm + L::s_col(step) + col0, pk);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars->s_done[L::s_buf(step)]);
        if (!(ok = warp_wait(&bars->dp_full[L::dp_buf(step)], L::dp_par(step), bars, 0x3306))) break;
        tc_fence_after_sync();
        uint32_t rr[32], ds[16];
        const uint32_t dp = tm + L::dp_col(step) + col0;
        tmem_ld(dp, rr);
        tc_fence_before_sync();
        mbar_arrive(&bars->dp_read[L::dp_buf(step)]);
        const float4* d4 = reinterpret_cast<const float4*>(nlse + 64 + col0);
#pragma unroll
        for (int e4 = 0; e4 < 8; ++e4) {
          const float4 dd = d4[e4];
          const float2 ds01 = __fmul2_rn(
              make_float2(__uint_as_float(pr[4 * e4]), __uint_as_float(pr[4 * e4 + 1])),
              __fadd2_rn(make_float2(__uint_as_float(rr[4 * e4]), __uint_as_float(rr[4 * e4 + 1])),
                         make_float2(dd.x, dd.y)));
          const float2 ds23 = __fmul2_rn(
              make_float2(__uint_as_float(pr[4 * e4 + 2]), __uint_as_float(pr[4 * e4 + 3])),
              __fadd2_rn(make_float2(__uint_as_float(rr[4 * e4 + 2]), __uint_as_float(rr[4 * e4 + 3])),
                         make_float2(dd.z, dd.w)));
          ds[2 * e4] = pack_bf16x2(ds01.x, ds01.y);
          ds[2 * e4 + 1] = pack_bf16x2(ds23.x, ds23.y);
        }
        tmem_st16(tm + L::s_col(step) + col0 + 16, ds);
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars->ds_ready[L::s_buf(step)]);
        if (++tile == first + per) tile = first;
      }
      if (!ok) break;
      pending = true;
      pending_k = at_k;
      pending_v = at_v;
      nb += n;
      ++tl;
    }
  }
  bwd_teardown(bars, warp, tmem, 0x32ff);
}

// Items of a launch as CTAs, at most one an SM.
unsigned grid_of(long long items, int sms) { return static_cast<unsigned>(std::min<long long>(items, sms)); }

template <int D, bool CAUSAL, int DP_SMEM>
cudaError_t launch_dq(const BwdParams& p, long long items, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> ready;
  return launch_behind(fa_packed_dq_kernel<D, CAUSAL, DP_SMEM>, p, grid_of(items, sms), kDqThreads,
                       DqLayout<D, DP_SMEM>::kSmem, ready, s);
}
template <int D, bool CAUSAL, int DP_SMEM>
cudaError_t launch_dkdv(const BwdParams& p, long long items, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> ready;
  return launch_behind(fa_packed_dkdv_kernel<D, CAUSAL, DP_SMEM>, p, grid_of(items, sms), kDkThreads,
                       DkLayout<D, DP_SMEM>::kSmem, ready, s);
}

// DP_SMEM at d = 128, by the steps that an item has on average.  Where they are few, it counts for more that
// shared memory is free at once for the next item's tensors (1), which then arrive while this one's products
// run, than a second buffer of scores (2).  Measured: 400 samples of 64 tokens, 32 heads on 8, one step an item of
// dq, 156 us with 1 and 175 with 2; 300 of 65 to 100 tokens, 16 on 16, 173 and 166; two of 8192, 1960 and 1330.
// dk and dv: 100 samples of 256 tokens, 16 on 16, four steps at most, 136 and 148; 300 of 65 to 100, 32 on 8, up
// to seven, 147 and 140; two of 8192, 2042 and 1298.
constexpr int kShortDq = 1, kShortDk = 4;

}  // namespace

cudaError_t launch_backward_packed(const PackedArgs& a, const CUtensorMap* maps, cudaStream_t s) {
  g_packed_bwd_used.store(true, std::memory_order_release);
  const int Hq = a.q.heads, Hkv = a.k.heads;
  const PackedTiling t = packed_tiling(Hq, Hkv);
  const PackedLayout l = packed_layout(a.B, a.total_q, a.total_k, Hq, Hkv, true);
  const bool dq_short = a.total_k <= 64ll * kShortDq * a.B;
  const bool dk_short = 1ll * a.total_q * t.per_kv <= 1ll * t.TT64 * kShortDk * a.B;
  cudaError_t e = launch_packed_plan(a, maps, 4, true, s);
  if (e != cudaSuccess) return e;
  char* ws = static_cast<char*>(a.workspace);
  auto out = [](const HeadsView& v) { return static_cast<__nv_bfloat16*>(const_cast<void*>(v.p)); };
  BwdParams p{};
  p.header = reinterpret_cast<PackedHeader*>(ws);
  p.maps = reinterpret_cast<const CUtensorMap*>(ws + l.maps);
  p.lse = a.lse;
  p.D = reinterpret_cast<float*>(ws + l.D);
  p.o = out(a.o), p.o_token = a.o.token, p.o_head = a.o.head;
  p.dO = out(a.dO), p.dO_token = a.dO.token, p.dO_head = a.dO.head;
  p.dq = out(a.dq), p.dq_token = a.dq.token, p.dq_head = a.dq.head;
  p.dk = out(a.dk), p.dk_token = a.dk.token, p.dk_head = a.dk.head;
  p.dv = out(a.dv), p.dv_token = a.dv.token, p.dv_head = a.dv.head;
  p.total_q = a.total_q;
  p.P = t.P;
  p.TT = 2 * t.TT64;
  p.TT64 = t.TT64;
  p.heads = t.heads;
  p.per_kv = t.per_kv;
  p.Hkv = Hkv;
  p.scale = a.scale;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  // the dq kernel streams keys and values, the other the queries and dO of a group's heads
  p.list = reinterpret_cast<const PackedEntry*>(ws + l.list[0]);
  const long long qi = a.total_q > 0 ? (a.total_q / p.TT + static_cast<long long>(a.B)) * t.heads : 0;
  p.chunk = packed_chunk(a.total_k, a.d, Hkv, qi, a.num_sms) * t.per_kv;
  if (a.d == 64)
    e = a.causal ? launch_dq<64, true, 1>(p, qi, a.num_sms, s) : launch_dq<64, false, 1>(p, qi, a.num_sms, s);
  else if (dq_short)
    e = a.causal ? launch_dq<128, true, 1>(p, qi, a.num_sms, s) : launch_dq<128, false, 1>(p, qi, a.num_sms, s);
  else
    e = a.causal ? launch_dq<128, true, 2>(p, qi, a.num_sms, s) : launch_dq<128, false, 2>(p, qi, a.num_sms, s);
  if (e != cudaSuccess) return e;
  p.list = reinterpret_cast<const PackedEntry*>(ws + l.list[1]);
  const long long ki = a.total_k > 0 ? (a.total_k / 128ll + a.B) * Hkv : 0;
  p.chunk = packed_chunk(static_cast<long long>(a.total_q) * (Hq / Hkv), a.d, Hkv, ki, a.num_sms);
  if (a.d == 64)
    return a.causal ? launch_dkdv<64, true, 1>(p, ki, a.num_sms, s) : launch_dkdv<64, false, 1>(p, ki, a.num_sms, s);
  if (dk_short)
    return a.causal ? launch_dkdv<128, true, 1>(p, ki, a.num_sms, s) : launch_dkdv<128, false, 1>(p, ki, a.num_sms, s);
  return a.causal ? launch_dkdv<128, true, 2>(p, ki, a.num_sms, s) : launch_dkdv<128, false, 2>(p, ki, a.num_sms, s);
}

cudaError_t packed_bwd_read_clear_error(uint32_t* out, cudaStream_t s) {
  *out = 0;
  if (!g_packed_bwd_used.load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  uint32_t v = 0;
  e = cudaMemcpyFromSymbol(&v, g_packed_bwd_error, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_packed_bwd_error, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}

}  // namespace fa
