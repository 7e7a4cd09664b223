// fa_packed.cu — the plan of attention over packed sequences, and its forward kernel.
//
// The forward kernel is the pipeline of fa_fwd.cu over the items of the plan: two 128-row
// query tiles stay in shared memory while 128-row key and value tiles stream through a ring; S =
// Q K^T and O += P V on the tensor core with S, P and O in tensor memory; one softmax thread
// a row, with a running maximum that moves only when a row needs it. The next item's tiles are
// copied while one's products run.
//
// Bound by the tensor core at d = 128: two causal sequences of 8192, 32 heads on 8, take 640 us on a
// cool GPU, 1.72 PFLOP/s of the triangle, and 710 us in a loop, under the power limit. 24 prompts
// of 1 to 2048 tokens take 250 us: 21 items a CTA, whose starts and ends take 2.7 us each (the tiles themselves are
// 90 % useful). At d = 64 the
// products are half as long, and the chain S, softmax, P V of a tile is what takes the time: 31
// sequences of up to 1500 tokens, 16 heads on 2, full, take 116 us with the tensor core busy for
// 40 % of them, and 64 causal samples of up to 512 tokens, 12 heads, 48 us.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "fa_packed.cuh"
#include "sm103_ptx.cuh"

namespace fa {
namespace {

__device__ unsigned int g_packed_error;
// Set by the first launch: until then the record above is clean and need not be copied, which takes 10 us.
std::atomic<bool> g_packed_used{false};

// ============================================================ plan
constexpr int kPlanThreads = 1024;
constexpr int kBuckets = 1024;

struct Span {
  int q0, n, k0, m;
};

__device__ __forceinline__ int within(int x, int hi) { return min(max(x, 0), hi); }

__device__ __forceinline__ Span span_of(const PackedPlanArgs& a, int b) {
  Span s;
  s.q0 = within(a.cu_q[b], a.total_q);
  s.n = max(within(a.cu_q[b + 1], a.total_q) - s.q0, 0);
  s.k0 = within(a.cu_k[b], a.total_k);
  s.m = max(within(a.cu_k[b + 1], a.total_k) - s.k0, 0);
  return s;
}

// Bucket of tile t of a list: list 0 counts a query tile's key tiles, list 1 a key tile's
// query tiles.
__device__ __forceinline__ int bucket_of(const PackedPlanArgs& a, int which, const Span& s, int t) {
  int cost;
  if (which == 0) {
    const int last = min(s.n, (t + 1) * a.q_span) - 1;
    cost = (packed_keys(last, s.n, s.m, a.causal) + 127) >> 7;
  } else {
    // the first query that sees the tile's first key
    const int first = a.causal ? max(t * a.k_span - (s.m - s.n), 0) : 0;
    cost = s.n > first ? (s.n + a.TT64 - 1) / a.TT64 - first / a.TT64 : 0;
  }
  return min(cost >> a.shift[which], kBuckets - 1);
}

// Block b < nlists builds list b: a counting sort of all tiles by bucket, longest first
// (the order within a bucket is that of the atomics; results do not depend on it).  The
// other blocks write tensor maps, a thread each.  A warp takes up to 32 sequences at a time
// (few enough that all warps have some): their spans in one load each, then sequence by
// sequence with a lane a tile.
__global__ void __launch_bounds__(kPlanThreads) fa_packed_plan_kernel(const __grid_constant__ PackedPlanArgs a) {
  grid_dependency_launch();
  if (blockIdx.x >= static_cast<unsigned>(a.nlists)) {
    const long long i = static_cast<long long>(blockIdx.x - a.nlists) * kPlanThreads + threadIdx.x;
    const int b = static_cast<int>(i / a.nmaps), t = static_cast<int>(i - static_cast<long long>(b) * a.nmaps);
    if (b >= a.B) return;
    const Span s = span_of(a, b);
    const bool keys = t == 1 || t == 2;
    CUtensorMap* out = a.maps + i;
    const uint4* src = reinterpret_cast<const uint4*>(&a.map[t]);
    uint4* dst = reinterpret_cast<uint4*>(out);
#pragma unroll
    for (int w = 0; w < 8; ++w) dst[w] = src[w];
    const uint64_t at = reinterpret_cast<uint64_t>(a.base[t] + (keys ? s.k0 : s.q0) * a.token[t]);
    const uint32_t len = static_cast<uint32_t>(max(keys ? s.m : s.n, 1));
    asm volatile("tensormap.replace.tile.global_address.global.b1024.b64 [%0], %1;" ::"l"(out), "l"(at)
                 : "memory");
    if (keys) {  // (d, tokens, heads)
      asm volatile(
          "tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;\n\t"
          "tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 2, %2;" ::"l"(out),
          "r"(len), "r"(a.Hkv)
          : "memory");
    } else {  // (d, heads of a tile, tokens, head groups)
      asm volatile(
          "tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 1, %1;\n\t"
          "tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 2, %2;\n\t"
          "tensormap.replace.tile.global_dim.global.b1024.b32 [%0], 3, %3;" ::"l"(out),
          "r"(a.P), "r"(len), "r"(a.groups)
          : "memory");
    }
    asm volatile("fence.proxy.tensormap::generic.release.gpu;" ::: "memory");
    return;
  }
  __shared__ unsigned hist[kBuckets];
  __shared__ unsigned warp_sum[32];
  const int which = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kBuckets; i += kPlanThreads) hist[i] = 0;
  __syncthreads();
  // every tile in turn: f(bucket, sequence, span, tile)
  auto tiles = [&](auto&& f) {
    const int each = min((a.B + kPlanThreads / 32 - 1) / (kPlanThreads / 32), 32);
    for (int b0 = warp * each; b0 < a.B; b0 += each * (kPlanThreads / 32)) {
      Span mine = {0, 0, 0, 0};
      if (lane < each && b0 + lane < a.B) mine = span_of(a, b0 + lane);
      const int own = which == 0 ? (mine.n + a.q_span - 1) / a.q_span : (mine.m + a.k_span - 1) / a.k_span;
      unsigned left = __ballot_sync(0xffffffffu, own > 0);
      while (left) {
        const int src = __ffs(left) - 1;
        left &= left - 1;
        Span s;
        s.q0 = __shfl_sync(0xffffffffu, mine.q0, src);
        s.n = __shfl_sync(0xffffffffu, mine.n, src);
        s.k0 = __shfl_sync(0xffffffffu, mine.k0, src);
        s.m = __shfl_sync(0xffffffffu, mine.m, src);
        const int nt = __shfl_sync(0xffffffffu, own, src);
        for (int t = lane; t < nt; t += 32) f(bucket_of(a, which, s, t), b0 + src, s, t);
        __syncwarp();
      }
    }
  };
  tiles([&](int k, int, const Span&, int) { atomicAdd(&hist[k], 1u); });
  __syncthreads();
  // entries before each bucket, the longest first (one bucket a thread)
  const int k = kBuckets - 1 - threadIdx.x;
  const unsigned own = hist[k];
  unsigned x = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sum[warp] = x;
  __syncthreads();
  if (warp == 0) {
    unsigned y = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    warp_sum[lane] = y;
  }
  __syncthreads();
  const unsigned before = x - own + (warp > 0 ? warp_sum[warp - 1] : 0u);
  hist[k] = before;
  if (threadIdx.x == kPlanThreads - 1) {
    a.header->next[which] = 0;
    a.header->count[which] = min(before + own, a.most[which]);
  }
  __syncthreads();
  tiles([&](int bucket, int b, const Span& s, int t) {
    const unsigned at = atomicAdd(&hist[bucket], 1u);
    if (at < a.most[which]) {  // (starts that descend can list more tiles than there are)
      int4* p = reinterpret_cast<int4*>(a.list[which] + at);
      p[0] = make_int4(b, t, s.q0, s.n);
      p[1] = make_int4(s.k0, s.m, 0, 0);
    }
  });
}
static_assert(kBuckets == kPlanThreads, "one bucket a thread in the scan");

// ============================================================ forward
constexpr int kFwdThreads = 352;  // two softmax warpgroups, a TMA and two MMA warps
constexpr int kTmaWarp = 8;
constexpr int kMmaWarp = 9;
constexpr int kMaxStages = 4;
constexpr float kLn2 = 0.69314718055994530942f;
// As in fa_fwd.cu: the running maximum moves when a tile's exceeds it by 2^8, and a tile taken
// against the old one stands while a row's sum of P is at most 2^16 (bf16 rounds
// relative to the value, and O and l carry the same factor).
constexpr float kLazyRescaleLog2 = 8.0f;
constexpr float kSpeculateSumBound = 65536.0f;

template <int D>
struct FwdLayout {
  static constexpr int kChunks = D / 64;
  static constexpr uint32_t kTileBytes = 128u * D * 2;
  static constexpr int kStages = D == 64 ? 4 : 2;  // key and value tiles under way, as many as fit
  // Two Q tiles, and room for one or both of the next item's, copied while this one's products run
  // (at d = 128, 24 prompts of up to 2048 tokens take 259 us, and 268 with two Q tiles in all).
  static constexpr int kQTiles = D == 64 ? 4 : 3;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + kQTiles * kTileBytes;
  static constexpr uint32_t kV = kK + kStages * kTileBytes;
  static constexpr uint32_t kBar = kV + kStages * kTileBytes;
  static constexpr uint32_t kSmemUsed = kBar + 1024 + 1024;  // + align slack
  // at least 116 KB, so two CTAs never share an SM (each takes all 512 TMEM columns)
  static constexpr uint32_t kSmem = kSmemUsed > 118784u ? kSmemUsed : 118784u;
  static constexpr uint32_t kTmemCols = 512;  // S0, S1, O0, O1
  __host__ __device__ static constexpr uint32_t s_col(int g) { return 128u * g; }
  __host__ __device__ static constexpr uint32_t o_col(int g) { return 256u + D * g; }
};

struct FwdBars {
  // Q tiles. Copied: by group, for its tile number t at t % 4, so that a group sees every phase of its
  // barriers and none twice (four tiles at most are unread). The S products that read it are done: by slot.
  uint64_t q_full[2][4], q_empty[4];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages];
  uint64_t v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t s_full[2], p_ready[2], pv_done[2];
  uint64_t item_full[kPackedRing], item_empty[kPackedRing];
  uint64_t turn[2];    // the other tile's products of a step are issued
  uint64_t o_free[2];  // softmax warpgroup g has read its O for the epilogue
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  PackedItem item[kPackedRing];
};
static_assert(sizeof(FwdBars) <= 1024, "barrier block overruns its shared memory");

struct FwdParams {
  PackedHeader* header;
  const PackedEntry* list;
  const CUtensorMap* maps;  // three a sequence: q, k, v
  __nv_bfloat16* o;
  long long o_token, o_head;
  float* lse;
  int total_q;
  int P, TT, heads, per_kv, chunk;
  float scale_log2;
  int causal;
};

// A wait's loop out of line: the code of the kernel stays small.
__device__ __noinline__ bool wait_loop(uint64_t* bar, uint32_t par, FwdBars* b, uint32_t code) {
  return mbar_wait(bar, par, &b->abort_flag, &g_packed_error, code);
}
__device__ __forceinline__ bool bar_wait(uint64_t* bar, uint32_t par, FwdBars* b, uint32_t code) {
  return mbar_try_wait(smem_u32(bar), par) || wait_loop(bar, par, b, code);
}
// The same by a whole warp, with one answer.
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t par, FwdBars* b, uint32_t code) {
  return __all_sync(0xffffffffu, bar_wait(bar, par, b, code));
}

template <int D>
__device__ __forceinline__ int ring_slot(int pos) {
  return static_cast<int>(static_cast<unsigned>(pos) % FwdLayout<D>::kStages);
}
template <int D>
__device__ __forceinline__ uint32_t ring_phase(int pos) {
  return (static_cast<unsigned>(pos) / FwdLayout<D>::kStages) & 1u;
}

// Key tiles that query tile 2 * pair + g of an item goes through.
__device__ __forceinline__ int item_tiles(const PackedItem& it, int g, int TT, bool causal) {
  const int first = (2 * it.e.tile + g) * TT;
  if (first >= it.e.n) return 0;
  return (packed_keys(min(first + TT, it.e.n) - 1, it.e.n, it.e.m, causal) + 127) >> 7;
}

template <int D, bool CAUSAL>
__global__ void __launch_bounds__(kFwdThreads, 1) fa_packed_fwd_kernel(const __grid_constant__ FwdParams p) {
  using L = FwdLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  FwdBars* bars = reinterpret_cast<FwdBars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 2);  // the two MMA warps
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars->q_full[0][i], 1);
      mbar_init(&bars->q_full[1][i], 1);
      mbar_init(&bars->q_empty[i], 1);
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&bars->s_full[g], 1);
      mbar_init(&bars->p_ready[g], 128);
      mbar_init(&bars->pv_done[g], 1);
      mbar_init(&bars->o_free[g], 128);
      mbar_init(&bars->turn[g], 1);
    }
    for (int r = 0; r < kPackedRing; ++r) {
      mbar_init(&bars->item_full[r], 1);
      mbar_init(&bars->item_empty[r], 258);  // the softmax threads and the MMA warps
    }
    mbar_init(&bars->drain, 2);
    bars->abort_flag = (*static_cast<volatile unsigned int*>(&g_packed_error) != 0) ? 1 : 0;
    fence_mbar_init();
  }
  // rows that no box fills stay zero
  if (p.P * p.TT < 128) {
    for (uint32_t i = threadIdx.x; i < L::kQTiles * L::kTileBytes / 16; i += kFwdThreads)
      reinterpret_cast<uint4*>(smem + L::kQ)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  __syncthreads();
  if (bars->abort_flag) return;
  if (warp == kMmaWarp) {
    tmem_alloc(&bars->tmem_base, L::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  grid_dependency_wait();

  if (warp == kTmaWarp) {
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      auto wait = [&](uint64_t* bar, uint32_t par, uint32_t code) {
        return bar_wait(bar, par, bars, code);
      };
      const uint32_t q_bytes = static_cast<uint32_t>(p.P * p.TT) * 128u * L::kChunks;
      int kvb = 0, qc = 0, qt[2] = {0, 0};  // K / V tiles, Q tiles, Q tiles of a group so far
      PackedItem it = packed_claim(p.header, p.list, 0, p.heads, p.chunk);
      for (int t = 0;; ++t) {
        const int r = t % kPackedRing;
        if (!wait(&bars->item_empty[r], ((t / kPackedRing) & 1) ^ 1, 0x1104)) break;
        bars->item[r] = it;
        mbar_arrive(&bars->item_full[r]);
        if (it.head < 0) break;
        const int n0 = item_tiles(it, 0, p.TT, CAUSAL), n1 = item_tiles(it, 1, p.TT, CAUSAL);
        const int nmax = max(n0, n1);
        if (nmax == 0) {
          it = packed_claim(p.header, p.list, 0, p.heads, p.chunk);
          continue;
        }
        const CUtensorMap* maps = p.maps + 3ll * it.e.seq;
        tensormap_acquire(maps);
        tensormap_acquire(maps + 1);
        tensormap_acquire(maps + 2);
        const int kh = it.head / p.per_kv, qh = it.head, pair = it.e.tile;
        auto load_q = [&](int g) {
          if ((g ? n1 : n0) == 0) return true;
          const int slot = qc % L::kQTiles;
          if (!wait(&bars->q_empty[slot], ((qc / L::kQTiles) & 1) ^ 1, 0x1103)) return false;
          uint64_t* full = &bars->q_full[g][qt[g]++ & 3];
          mbar_arrive_expect_tx(full, q_bytes);
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c)
            tma_load_4d(smem + L::kQ + slot * L::kTileBytes + c * 16384, maps, full, c * 64, 0,
                        (2 * pair + g) * p.TT, qh);
          ++qc;
          return true;
        };
        PackedItem next = it;
        bool ok = load_q(0);
        for (int j = 0; ok && j < nmax; ++j) {
          const int s = ring_slot<D>(kvb + j);
          const uint32_t ph = ring_phase<D>(kvb + j);
          if (!(ok = wait(&bars->k_empty[s], ph ^ 1, 0x1101))) break;
          mbar_arrive_expect_tx(&bars->k_full[s], L::kTileBytes);
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c)
            tma_load_3d(smem + L::kK + s * L::kTileBytes + c * 16384, maps + 1, &bars->k_full[s], c * 64,
                        j * 128, kh);
          if (j == 0 && !(ok = load_q(1))) break;
          if (!(ok = wait(&bars->v_empty[s], ph ^ 1, 0x1102))) break;
          mbar_arrive_expect_tx(&bars->v_full[s], L::kTileBytes);
#pragma unroll
          for (int c = 0; c < L::kChunks; ++c)
            tma_load_3d(smem + L::kV + s * L::kTileBytes + c * 16384, maps + 2, &bars->v_full[s], c * 64,
                        j * 128, kh);
          // the next item is asked for while the last two tiles are under way
          if (j == max(nmax - 2, 0)) next = packed_claim(p.header, p.list, 0, p.heads, p.chunk);
        }
        if (!ok) break;
        kvb += nmax;
        it = next;
      }
    }
    __syncwarp();
  } else if (warp >= kMmaWarp) {
    // ------------------------------------------------ MMA issuers, one a query tile
    // Issuing is what the tensor core waited for: 8 products take 210 to 290 cycles to issue, a
    // commit 50, a wait that is over 70, against 512 cycles that 8 products of 128 columns run.
    // So each query tile has a warp of its own, which waits while the other issues; they take
    // turns, because products of both in flight at once would end later for both, and their
    // softmaxes would meet.  The whole warp runs the loop on values that are the same in all
    // lanes, so that descriptors lie in uniform registers, where the instruction wants them;
    // one elected lane issues.
    const int g = warp - kMmaWarp;
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, 128, false, false);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true);
    const uint32_t tm = uniform(tmem), sc = tm + uniform(L::s_col(g)), oc = tm + uniform(L::o_col(g));
    const uint32_t sQ = uniform(smem_u32(smem + L::kQ));
    uint32_t qbase = sQ;
    const uint32_t sK = uniform(smem_u32(smem + L::kK)), sV = uniform(smem_u32(smem + L::kV));
    auto wait = [&](uint64_t* bar, uint32_t par, uint32_t code) { return all_wait(bar, par, bars, code); };
    auto issue_s = [&](int slot) {
      const uint32_t kbase = sK + slot * L::kTileBytes;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
        umma_ss(sc, sdesc_sw128(qbase + off, 16, 1024), sdesc_sw128(kbase + off, 16, 1024), idesc_qk,
                kk > 0 ? 1u : 0u);
      }
      umma_commit(&bars->s_full[g]);
      umma_commit(&bars->k_empty[slot]);
    };
    auto issue_pv = [&](int slot, bool first) {
      const uint32_t vbase = sV + slot * L::kTileBytes;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        umma_ts(oc, sc + kk * 8, sdesc_sw128(vbase + kk * 2048, 16384, 1024), idesc_pv, (!first || kk > 0) ? 1u : 0u);
      umma_commit(&bars->v_empty[slot]);
    };
    // For key tile j: PV_j and S_{j+1}.  A query tile may have no work in an item (it lies
    // behind the sequence, or sees no key), or end before the other: it then gives the
    // copied tiles back unread.
    int kvb = 0, qc = 0, qt = 0, base = 0, used = 0, turns = 0;
    auto turn = [&]() {  // (the first tile's warp goes first)
      const uint32_t par = static_cast<uint32_t>(turns++ & 1) ^ (g == 0 ? 1u : 0u);
      return wait(&bars->turn[g], par, 0x120c);
    };
    for (int t = 0;; ++t) {
      const int r = t % kPackedRing;
      if (!wait(&bars->item_full[r], (t / kPackedRing) & 1, 0x120b)) break;
      const PackedItem it = bars->item[r];
      __syncwarp();
      if (elect_one()) mbar_arrive(&bars->item_empty[r]);
      if (uniform(it.head) < 0) break;
      const int n0 = uniform(item_tiles(it, 0, p.TT, CAUSAL)), n1 = uniform(item_tiles(it, 1, p.TT, CAUSAL));
      const int n = g == 0 ? n0 : n1, nmax = max(n0, n1);
      if (nmax == 0) continue;
      const int slot = (qc + (g == 1 && n0 > 0 ? 1 : 0)) % L::kQTiles;
      qbase = sQ + slot * L::kTileBytes;
      if ((n > 0 && !wait(&bars->q_full[g][qt & 3], (qt >> 2) & 1, 0x1201)) ||
          !wait(&bars->k_full[ring_slot<D>(kvb)], ring_phase<D>(kvb), 0x1202) || !turn())
        break;
      tc_fence_after_sync();
      if (elect_one()) {
        if (n > 0)
          issue_s(ring_slot<D>(kvb));
        else
          mbar_arrive(&bars->k_empty[ring_slot<D>(kvb)]);
        if (n == 1) umma_commit(&bars->q_empty[slot]);
        mbar_arrive(&bars->turn[1 - g]);
      }
      __syncwarp();
      bool ok = true;
      // At d = 64 the turn is taken before P is waited for, so that one wait fewer follows P (31
      // sequences of up to 1500 tokens, 16 heads on 2, full, with two key and value tiles under way: 125
      // us, and 131 the other way round; with four 118); at d = 128, where the products take
      // longer than the waits, that other way is 1 to 2 % faster.
      auto p_wait = [&](int j) { return j >= n || wait(&bars->p_ready[g], (base + j) & 1, 0x1203); };
#pragma unroll 1
      for (int j = 0; j < nmax; ++j) {
        const int pos = kvb + j, s = ring_slot<D>(pos), sn = ring_slot<D>(pos + 1);
        ok = wait(&bars->v_full[s], ring_phase<D>(pos), 0x1204) &&
             (j > 0 || n == 0 || used == 0 || wait(&bars->o_free[g], (used - 1) & 1, 0x1209)) &&
             (j + 1 >= nmax || wait(&bars->k_full[sn], ring_phase<D>(pos + 1), 0x1205)) &&
             (D == 64 ? turn() && p_wait(j) : p_wait(j) && turn());
        if (!ok) break;
        tc_fence_after_sync();
        if (elect_one()) {
          if (j < n)
            issue_pv(s, j == 0);
          else
            mbar_arrive(&bars->v_empty[s]);
          if (j + 1 == n) umma_commit(&bars->pv_done[g]);
          if (j + 1 < n)
            issue_s(sn);
          else if (j + 1 < nmax)
            mbar_arrive(&bars->k_empty[sn]);
          if (j + 2 == n) umma_commit(&bars->q_empty[slot]);
          mbar_arrive(&bars->turn[1 - g]);
        }
        __syncwarp();
      }
      if (!ok) break;
      qt += n > 0;
      qc += (n0 > 0) + (n1 > 0);
      kvb += nmax;
      base += n;
      used += n > 0;
    }
    __syncwarp();
    if (elect_one()) umma_commit(&bars->drain);
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax warpgroups
    const int g = warp >> 2;          // which query tile of the pair
    const int t = threadIdx.x & 127;  // row within the tile, TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t scol = tmem + lane_off + L::s_col(g), ocol = tmem + lane_off + L::o_col(g);
    auto warp_wait = [&](uint64_t* bar, uint32_t par, uint32_t code) { return all_wait(bar, par, bars, code); };
    int tb = 0, used = 0;  // key tiles of earlier items, and items with any
    for (int ti = 0;; ++ti) {
      const int r = ti % kPackedRing;
      if (!warp_wait(&bars->item_full[r], (ti / kPackedRing) & 1, 0x1304)) break;
      // (what only the end of the item wants is read again there: with it the loop over key tiles
      // spills, and 24 prompts of up to 2048 tokens take 259 us, not 250)
      int nkv, tok0, m, off;
      {
        const PackedItem it = bars->item[r];
        if (it.head < 0) break;
        nkv = item_tiles(it, g, p.TT, CAUSAL);
        tok0 = (2 * it.e.tile + g) * p.TT;
        m = it.e.m;
        off = m - it.e.n;  // causal: keys j <= tok + off
      }
      const int tok = tok0 + t / p.P;
      float m_run = -INFINITY;  // running (lazily moved) max of s * scale * log2(e)
      float l_run = 0.0f;
      bool ok = true;
      for (int j = 0; j < nkv; ++j) {
        if (!(ok = warp_wait(&bars->s_full[g], (tb + j) & 1, 0x1301))) break;
        tc_fence_after_sync();
        uint32_t sr[128];
        const int kv0 = j * 128;
        const bool need_mask = (CAUSAL && kv0 + 127 > tok0 + off) || kv0 + 128 > m;
        auto load_scores = [&]() {
          tmem_ld32(scol + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
          tmem_ld32(scol + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
          tmem_ld32(scol + 64, *reinterpret_cast<uint32_t(*)[32]>(&sr[64]));
          tmem_ld32(scol + 96, *reinterpret_cast<uint32_t(*)[32]>(&sr[96]));
          tmem_ld_wait();
          reg_pin(sr);
          if (need_mask) {
            const int lim = (CAUSAL ? min(tok + off, m - 1) : m - 1) - kv0;  // columns <= lim are seen
#pragma unroll
            for (int c = 0; c < 128; ++c)
              if (c > lim) sr[c] = __float_as_uint(-INFINITY);
          }
        };
        load_scores();
        float sum = 0.0f;
        auto exp_tile = [&]() {
          const float m_use = (m_run == -INFINITY) ? 0.0f : m_run;
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2), nm2 = make_float2(-m_use, -m_use);
          float2 sp[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                          make_float2(0.f, 0.f)};  // partial row sums
#pragma unroll
          for (int c = 0; c < 64; ++c) {
            const float2 x = __ffma2_rn(
                make_float2(__uint_as_float(sr[2 * c]), __uint_as_float(sr[2 * c + 1])), sc2, nm2);
            const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sp[c & 3] = __fadd2_rn(sp[c & 3], e);
            sr[c] = pack_bf16x2(e.x, e.y);
          }
          const float2 s4 = __fadd2_rn(__fadd2_rn(sp[0], sp[1]), __fadd2_rn(sp[2], sp[3]));
          sum = s4.x + s4.y;
        };
        bool move = false;
        float alpha = 1.0f;
        bool exact = !__all_sync(0xffffffffu, m_run != -INFINITY);
        // once, or twice where the first pass, against the old maximum, leaves its bound
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          if (exact) {
            const float m_blk = row_max128(sr) * p.scale_log2;
            move = __any_sync(0xffffffffu, m_blk > m_run + kLazyRescaleLog2);
            if (move) {
              const float m_new = fmaxf(m_run, m_blk);
              alpha = m_new == -INFINITY ? 1.0f : ex2_approx(m_run - m_new);  // 0 on the first tile
              l_run *= alpha;
              m_run = m_new;
            }
          }
          exp_tile();
          if (exact) break;
          if (!__any_sync(0xffffffffu, !(sum <= kSpeculateSumBound))) break;
          load_scores();  // the first pass overwrote sr with P
          exact = true;
        }
        tmem_st32(scol + 0, *reinterpret_cast<uint32_t(*)[32]>(&sr[0]));
        tmem_st32(scol + 32, *reinterpret_cast<uint32_t(*)[32]>(&sr[32]));
        if (move && j > 0) {
          // PV_g(j-1) completed before S_g(j) was reported, and PV_g(j) is not issued before
          // p_ready: O is stable here
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t rr[32];
            tmem_ld32(ocol + c * 32, rr);
            tmem_ld_wait();
            reg_pin(rr);
#pragma unroll
            for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st32(ocol + c * 32, rr);
          }
        }
        l_run += sum;
        tmem_st_wait();
        tc_fence_before_sync();
        mbar_arrive(&bars->p_ready[g]);
      }
      if (!ok) break;
      // ------------------------------------------------ epilogue
      const PackedItem it = bars->item[r];
      mbar_arrive(&bars->item_empty[r]);
      const bool stores = t < p.P * p.TT && tok < it.e.n;
      const int head = it.head * p.P + t % p.P;
      const long long off_o =
          stores ? static_cast<long long>(it.e.q0 + tok) * p.o_token + head * p.o_head : -1;
      if (nkv == 0) {
        // no key is seen: O = 0, lse = -inf (tensor memory is never read)
        if (stores) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + off_o);
#pragma unroll
          for (int e = 0; e < D / 8; ++e) dst[e] = make_uint4(0u, 0u, 0u, 0u);
          p.lse[static_cast<long long>(head) * p.total_q + it.e.q0 + tok] = -INFINITY;
        }
        continue;
      }
      tb += nkv;
      if (!warp_wait(&bars->pv_done[g], used++ & 1, 0x1303)) break;
      tc_fence_after_sync();
      // (a row whose keys all have a score of -inf is NaN, one that sees none is 0)
      const bool sees = !CAUSAL || tok + it.e.m >= it.e.n;
      const float inv_l = l_run > 0.0f ? 1.0f / l_run : (l_run == 0.0f ? (sees ? NAN : 0.0f) : l_run);
      // rows of this lane's 4-lane group are stored together, row by row
      long long dst[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) dst[k] = __shfl_sync(0xffffffffu, off_o, (lane & ~3) + k);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t rr[32], w[16];
        tmem_ld32(ocol + c * 32, rr);
        tmem_ld_wait();
        reg_pin(rr);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          w[e] = pack_bf16x2(__uint_as_float(rr[2 * e]) * inv_l, __uint_as_float(rr[2 * e + 1]) * inv_l);
        transpose_chunks<4>(w);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (dst[k] >= 0)
            *reinterpret_cast<uint4*>(p.o + dst[k] + c * 32 + (lane & 3) * 8) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
      }
      // O_g has been read: the next item's first P V may overwrite it
      tc_fence_before_sync();
      mbar_arrive(&bars->o_free[g]);
      if (stores)
        p.lse[static_cast<long long>(head) * p.total_q + it.e.q0 + tok] =
            l_run == 0.0f ? -INFINITY : (m_run + log2f(l_run)) * kLn2;
    }
  }

  // ------------------------------------------------ teardown
  if (warp == kMmaWarp) mbar_wait(&bars->drain, 0, &bars->abort_flag, &g_packed_error, 0x120f);
  if (bars->abort_flag) {
    // let any bulk copy already in flight land before the CTA exits
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kTmemCols);
  }
}

template <int D, bool CAUSAL>
cudaError_t launch_t(const FwdParams& p, unsigned blocks, cudaStream_t s) {
  static std::atomic<unsigned long long> ready;
  return launch_behind(fa_packed_fwd_kernel<D, CAUSAL>, p, blocks, kFwdThreads, FwdLayout<D>::kSmem, ready, s);
}

int bucket_shift(long long most) {
  int s = 0;
  while ((most >> s) >= kBuckets) ++s;
  return s;
}

}  // namespace

cudaError_t launch_packed_plan(const PackedArgs& a, const CUtensorMap* maps, int nmaps, bool backward,
                               cudaStream_t s) {
  const int Hq = a.q.heads, Hkv = a.k.heads;
  const PackedTiling t = packed_tiling(Hq, Hkv);
  const PackedLayout l = packed_layout(a.B, a.total_q, a.total_k, Hq, Hkv, backward);
  char* ws = static_cast<char*>(a.workspace);
  PackedPlanArgs p{};
  const HeadsView* views[4] = {&a.q, &a.k, &a.v, &a.dO};
  for (int i = 0; i < nmaps; ++i) {
    p.map[i] = maps[i];
    p.base[i] = static_cast<const __nv_bfloat16*>(views[i]->p);
    p.token[i] = views[i]->token;
  }
  p.nmaps = nmaps;
  p.P = t.P;
  p.groups = t.heads;
  p.Hkv = Hkv;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.B = a.B;
  p.total_q = a.total_q;
  p.total_k = a.total_k;
  p.causal = a.causal;
  p.q_span = 2 * (backward ? t.TT64 : t.TT);  // an entry of the forward pass is two tiles, each of 128 rows
  p.k_span = 128;
  p.TT64 = t.TT64;
  p.nlists = backward ? 2 : 1;
  p.most[0] = static_cast<unsigned>(a.total_q / p.q_span + a.B);
  p.most[1] = static_cast<unsigned>(a.total_k / p.k_span + a.B);
  p.shift[0] = bucket_shift(a.total_k / 128 + 1);
  p.shift[1] = bucket_shift(a.total_q / t.TT64 + 1);
  p.header = reinterpret_cast<PackedHeader*>(ws);
  p.maps = reinterpret_cast<CUtensorMap*>(ws + l.maps);
  for (int i = 0; i < 2; ++i) p.list[i] = reinterpret_cast<PackedEntry*>(ws + l.list[i]);
  const long long map_blocks = (static_cast<long long>(a.B) * nmaps + kPlanThreads - 1) / kPlanThreads;
  fa_packed_plan_kernel<<<static_cast<unsigned>(p.nlists + map_blocks), kPlanThreads, 0, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_forward_packed(const PackedArgs& a, const CUtensorMap* maps, cudaStream_t s) {
  g_packed_used.store(true, std::memory_order_release);
  const PackedTiling t = packed_tiling(a.q.heads, a.k.heads);
  const PackedLayout l = packed_layout(a.B, a.total_q, a.total_k, a.q.heads, a.k.heads, false);
  cudaError_t e = launch_packed_plan(a, maps, 3, false, s);
  if (e != cudaSuccess) return e;
  char* ws = static_cast<char*>(a.workspace);
  FwdParams p{};
  p.header = reinterpret_cast<PackedHeader*>(ws);
  p.list = reinterpret_cast<const PackedEntry*>(ws + l.list[0]);
  p.maps = reinterpret_cast<const CUtensorMap*>(ws + l.maps);
  p.o = static_cast<__nv_bfloat16*>(const_cast<void*>(a.o.p));
  p.o_token = a.o.token;
  p.o_head = a.o.head;
  p.lse = a.lse;
  p.total_q = a.total_q;
  p.P = t.P;
  p.TT = t.TT;
  p.heads = t.heads;
  p.per_kv = t.per_kv;
  p.scale_log2 = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634);
  p.causal = a.causal;
  const long long items = (a.total_q / (2ll * t.TT) + a.B) * t.heads;
  p.chunk = packed_chunk(a.total_k, a.d, a.k.heads, items, a.num_sms) * t.per_kv;
  const unsigned blocks = static_cast<unsigned>(std::min<long long>(items, a.num_sms));
  if (a.d == 64) return a.causal ? launch_t<64, true>(p, blocks, s) : launch_t<64, false>(p, blocks, s);
  return a.causal ? launch_t<128, true>(p, blocks, s) : launch_t<128, false>(p, blocks, s);
}

cudaError_t packed_read_clear_error(uint32_t* out, cudaStream_t s) {
  *out = 0;
  if (!g_packed_used.load(std::memory_order_acquire)) return cudaSuccess;
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  uint32_t v = 0;
  e = cudaMemcpyFromSymbol(&v, g_packed_error, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_packed_error, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}

}  // namespace fa
