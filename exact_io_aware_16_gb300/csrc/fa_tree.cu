// fa_tree.cu — attention of a tree of drafted tokens over the key/value cache
// (bf16 or e4m3), grouped heads, a length for each sequence.
//
// The G = Hq / Hkv query heads of a key head times the T drafts are R = G T
// query rows against one key/value sequence: o = softmax(scale q k^T) v over the
// committed tokens and the drafts that the row's mask names.  Every key and
// value is read once a row tile, and ~4 R FLOPs are done for each of its
// elements, so the step is bound by HBM up to a few dozen rows and the products
// run on the tensor core for all of them.
//
// Split.  The (sequence, key head) pairs are cut into tiles of KT keys and the
// list of all tiles into equal shares, one CTA a share (times the row tiles of
// 128 rows, which run side by side so that they read a key tile while it is in
// L2).  Lengths live on the device, so each CTA finds its share from lens
// itself.  A pair that one CTA covers is finished there; the partial results of
// the others ((m, l) and o, at most two a CTA) go to the workspace, and
// fa_tree_combine merges them by the running-maximum update.
//
// One CTA (two an SM, 256 tensor-memory columns each):
//   * warp 4 streams K and V tiles (and the scale bytes of an e4m3 cache)
//     through TMA rings;
//   * warp 5 issues S = Q K^T (M = 128 rows, N = KT keys) and O += P V;
//   * warps 0-3 own a tensor-memory lane a thread, a query row each: softmax, P
//     back into S's columns, epilogue.  Where R <= 64 the rows are repeated in the
//     lanes (REP = 2 or 4 times) and each copy takes 1 / REP of a tile's keys
//     with P = 0 elsewhere: all four warps work for any R, at no extra MMA, and
//     the copies are merged in the epilogue.
//
// e4m3 operands: kind::f8f6f4 takes the cache as it lies in memory.  Two e4m3
// pieces of 4 significant bits hold the 8 bits of a bf16 query exactly (its row
// scaled by a power of two into 448), and a probability to 2^-8: S and O
// accumulate both pieces, twice the MMAs at twice the bf16 rate.  The scales of
// keys and values join in the softmax: with e_j the exponent of value row j, the
// thread forms t_j = scale log2(e) 2^(k_j) S_j + e_j, keeps M = max t_j, and
// gives P_j = 2^(t_j - M) to the product with the codes, while the sum takes
// P_j 2^(-e_j); o = O / l needs no further factor.
#include <algorithm>
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

__device__ unsigned int g_tree_error;

constexpr int kTreeThreads = 192;
constexpr int kSoftThreads = 128;
constexpr int kTreeTmaWarp = 4;
constexpr int kTreeMmaWarp = 5;
constexpr uint32_t kTreeTmemCols = 256;  // S (and P) from column 0, O from 128
constexpr uint32_t kOCol = 128;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kScaleSlots = 4;

// A row's accumulator is rescaled only when its maximum grows by more than
// kLazy binades.  bf16 has the range for any P; the e4m3 pieces of P are scaled
// so that 2^kLazy times the largest P at the last rescale is still 448.
template <bool F8>
struct Lazy {
  static constexpr float kLog2 = F8 ? 2.0f : 8.0f;
  static constexpr float kPScaleLog2 = F8 ? 6.8073549220576f : 0.0f;  // log2(448 / 4)
};

template <int D, bool F8>
struct TreeLayout {
  static constexpr int kTile = F8 ? 128 : 64;              // keys a tile
  static constexpr uint32_t kRow = F8 ? D : 2 * D;         // bytes of a cache row
  static constexpr uint32_t kAtom = F8 && D == 64 ? 64 : 128;  // swizzle width in bytes
  static constexpr uint32_t kKvBytes = kTile * kRow;       // 16 KB (D = 128) or 8 KB
  static constexpr uint32_t kQChunk = 128u * kAtom;        // 128 rows of one atom
  static constexpr int kQChunks = F8 ? 2 : D / 64;         // e4m3: the two pieces
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kQ = 0;
  static constexpr uint32_t kK = kQ + kQChunks * kQChunk;
  static constexpr uint32_t kV = kK + kStages * kKvBytes;
  static constexpr uint32_t kScale = kV + kStages * kKvBytes;  // raw scale bytes, k then v
  static constexpr uint32_t kTable = kScale + (F8 ? kScaleSlots * 256u : 0u);
  static constexpr uint32_t kBar = kTable + (F8 ? 4u * 128u * 12u : 0u);
  static constexpr uint32_t kUsed = kBar + 2048 + 1024;  // + alignment slack
  // above a third of an SM's: never three CTAs (3 x 256 tensor-memory columns)
  static constexpr uint32_t kSmem = kUsed > 81920u ? kUsed : 81920u;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs an SM");
  // the epilogue's merge buffer (128 rows of 16 floats) lies over Q
  static_assert(kQChunks * kQChunk >= 128 * 64, "merge buffer fits");
};

struct TreeBars {
  uint64_t q_ready;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t sc_full[kScaleSlots], sc_empty[kScaleSlots];
  uint64_t s_full, p_ready, o_full, drain;
  uint32_t tmem_base;
  int abort_flag;
  unsigned int bad_lo, bad_hi;  // drafts whose value row holds NaN or infinities
  int start_b, start_h, start_t, count;  // this CTA's share
  int pair_tiles, pair_len;              // the pair at hand, as the softmax warps agree on it
  float row_m[kSoftThreads], row_l[kSoftThreads];
};
static_assert(sizeof(TreeBars) <= 2048, "barrier block");

struct TreeParams {
  const uint4* q;
  const int* lens;
  const unsigned long long* mask;
  long long mask_stride;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;     // [slots][prow][D]
  float2* part_ml;   // [slots][prow]
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const uint8_t* v;  // the value cache, for rows with NaN or infinities
  int B, Hkv, cap, G, T, R;
  int row_tiles, shares, prow;
  float scale_log2;
};

__device__ __forceinline__ bool t_wait(uint64_t* bar, uint32_t parity, TreeBars* b, uint32_t code) {
  return mbar_wait(bar, parity, &b->abort_flag, &g_tree_error, code);
}

// Keys of sequence b that exist: its committed tokens and its drafts.
__device__ __forceinline__ int seq_len(const TreeParams& p, int b) {
  return min(max(__ldg(p.lens + b), 0), p.cap);
}
__device__ __forceinline__ int seq_tiles(const TreeParams& p, int b, int tile) {
  return (min(seq_len(p, b) + p.T, p.cap) + tile - 1) / tile;
}

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Tiles of all (sequence, key head) pairs; the whole warp calls it.
__device__ __forceinline__ int all_tiles(const TreeParams& p, int tile) {
  int n = 0;
  for (int b = threadIdx.x & 31; b < p.B; b += 32) n += seq_tiles(p, b, tile);
  return warp_sum(n) * p.Hkv;
}

// Tiles a share: all shares but the last have this many.
__device__ __forceinline__ int share_size(int total, int shares) {
  return (total + shares - 1) / shares;
}

// A CTA's walk over the pairs that its share touches.
struct Walk {
  int b, h, t0, left;
  int n;       // tiles of this pair in the share
  int nt;      // tiles of the pair
  __device__ __forceinline__ Walk(const TreeBars* bars)
      : b(bars->start_b), h(bars->start_h), t0(bars->start_t), left(bars->count), n(0), nt(0) {}
  __device__ __forceinline__ bool valid(const TreeParams& p, int tile) {
    if (left <= 0) return false;
    set(seq_tiles(p, b, tile));
    return true;
  }
  __device__ __forceinline__ void set(int tiles) {
    nt = tiles;
    n = min(left, nt - t0);
  }
  __device__ __forceinline__ void next(const TreeParams& p) {
    left -= n;
    t0 = 0;
    if (++h == p.Hkv) {
      h = 0;
      ++b;
    }
  }
};

// ------------------------------------------------------------ tensor memory
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t* r) {
  static_assert(N == 16 || N % 32 == 0, "columns");
  if constexpr (N == 16) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  } else {
#pragma unroll
    for (int c = 0; c < N; c += 32)
      tmem_ld32(taddr + c, *reinterpret_cast<uint32_t(*)[32]>(r + c));
  }
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
               "r"(r[7])
               : "memory");
}

__device__ __forceinline__ void tmem_st8_zero(uint32_t taddr) {
  const uint32_t z = 0;
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1};" ::"r"(taddr),
               "r"(z)
               : "memory");
}

// ------------------------------------------------------------ conversions
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// Two fp32 as two e4m3 pieces each: hi = e4m3(x), lo = e4m3(x - hi).  The
// subtraction is exact in fp16 (both are multiples of x's fp16 unit, of at most
// 11 bits), x in fp16 is good to 2^-12.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const __nv_fp8x2_storage_t a =
      __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
  const __half2 back = __half2(__nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3));
  const __nv_fp8x2_storage_t b = __nv_cvt_halfraw2_to_fp8x2(
      static_cast<__half2_raw>(__hsub2(h, back)), __NV_SATFINITE, __NV_E4M3);
  hi = a;
  lo = b;
}

// Four fp32 as a word of high pieces and a word of low pieces.
__device__ __forceinline__ void split4(float x0, float x1, float x2, float x3, uint32_t& hi,
                                       uint32_t& lo) {
  uint32_t h0, l0, h1, l1;
  split2(x0, x1, h0, l0);
  split2(x2, x3, h1, l1);
  hi = h0 | (h1 << 16);
  lo = l0 | (l1 << 16);
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Address of 16-byte unit c of row r in a swizzled tile of `atom`-byte rows.
template <uint32_t ATOM>
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) {
  const uint32_t x = ATOM == 128 ? (c ^ (r & 7u)) : (c ^ ((r >> 1) & 3u));
  return r * ATOM + x * 16u;
}

// sdesc_sw128 with the swizzle of 64-byte rows (layout 4).
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t smem_addr, uint32_t lbo_bytes,
                                               uint32_t sbo_bytes) {
  return (sdesc_sw128(smem_addr, lbo_bytes, sbo_bytes) & ~(7ull << 61)) | (4ull << 61);
}
template <uint32_t ATOM>
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return ATOM == 128 ? sdesc_sw128(addr, lbo, sbo) : sdesc_sw64(addr, lbo, sbo);
}

// Bulk copy of plain bytes (both addresses 16-byte aligned, size a multiple of 16).
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------ query rows
// The thread's query row (row r of the pair, or zeros) into the swizzled
// operand, lane `lane`.  e4m3: two pieces of the row times 2^-e, the return
// value is e; bf16: as it is, returns 0.
template <int D, bool F8>
__device__ __forceinline__ int store_query(uint8_t* sq, const uint4* src, bool exists, int lane) {
  using L = TreeLayout<D, F8>;
  if constexpr (!F8) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      const uint4 x = exists ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      *reinterpret_cast<uint4*>(sq + (c >> 3) * L::kQChunk + swizzled<128>(lane, c & 7)) = x;
    }
    return 0;
  } else {
    uint4 x[D / 8];
    uint32_t m = 0;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      x[c] = exists ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
      m = __vmaxu2(m, finite_max8(x[c]));
    }
    const int e = scale_exponent(max(m & 0xffffu, m >> 16));
    const float s = pow2_of(-e);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4& y = x[2 * c + (i >> 1)];
        const uint32_t w0 = (i & 1) ? y.z : y.x, w1 = (i & 1) ? y.w : y.y;
        float f[4] = {bf_lo(w0), bf_hi(w0), bf_lo(w1), bf_hi(w1)};
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = fmaf(f[k], 0.0f, f[k] * s);  // infinities to NaN
        split4(f[0], f[1], f[2], f[3], hi[i], lo[i]);
      }
      const uint32_t at = swizzled<L::kAtom>(lane, c);
      *reinterpret_cast<uint4*>(sq + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(sq + L::kQChunk + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    return e;
  }
}

// ------------------------------------------------------------ value rows
// A tile that reaches past the committed tokens: value rows that no query row
// of the sequence sees become zero (P is zero there, but 0 * NaN is not), and
// in drafts that some row sees NaN and infinities become zero and the draft is
// noted: the epilogue adds them to the rows that see it.
template <int D, bool F8>
__device__ __forceinline__ void clean_values(uint8_t* sv, int kb0, int len, int end,
                                             unsigned long long any, TreeBars* bars) {
  using L = TreeLayout<D, F8>;
  constexpr int kParts = L::kRow / L::kAtom;             // 128-byte (or 64-byte) pieces a row
  static_assert(kParts * L::kTile <= kSoftThreads, "one piece a thread");
  const int c = threadIdx.x % L::kTile, part = threadIdx.x / L::kTile;
  if (part >= kParts) return;
  const int pos = kb0 + c;
  if (pos < len) return;
  const int j = pos - len;
  const bool live = pos < end && (any >> (j & 63) & 1);
  uint4* row = reinterpret_cast<uint4*>(sv + part * (L::kTile * L::kAtom) + c * L::kAtom);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < static_cast<int>(L::kAtom) / 16; ++i) {
    if (!live) {
      row[i] = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 x = row[i];
    uint32_t w[4] = {x.x, x.y, x.z, x.w}, hit = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t n = F8 ? __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu)
                            : __vcmpgeu2(w[k] & 0x7fff7fffu, 0x7f807f80u);
      hit |= n;
      w[k] &= ~n;
    }
    if (hit) {
      row[i] = make_uint4(w[0], w[1], w[2], w[3]);
      bad = true;
    }
  }
  if (bad) atomicOr(j < 32 ? &bars->bad_lo : &bars->bad_hi, 1u << (j & 31));
}

// ------------------------------------------------------------ softmax of a tile
struct RowState {
  float m, l;   // reference exponent (see Lazy) and sum
  float f;      // scale log2(e), times 2^e of the query row for e4m3
};

// One tile of S for this thread's row: CW columns from `c0` on.  Writes P, and
// rescales O (valid from the pair's second tile on).  table (e4m3): 2^k_j, e_j
// and 2^-e_j of those columns, 128 floats apart.
template <int D, bool F8, int REP>
__device__ __forceinline__ void softmax_tile(uint32_t tlane, int kq, RowState& st,
                                             const float* table, bool first, bool edge, int kb0,
                                             int len, int end, unsigned long long seen) {
  using L = TreeLayout<D, F8>;
  constexpr int CW = L::kTile / REP;
  const int c0 = kq * CW;
  uint32_t sr[CW];
  tmem_ld<CW>(tlane + c0, sr);
  tmem_ld_wait();
  reg_pin(sr);
#pragma unroll
  for (int c = 0; c < CW; c += 4) {
    if constexpr (F8) {
      const float4 k = *reinterpret_cast<const float4*>(table + c);
      const float4 e = *reinterpret_cast<const float4*>(table + 128 + c);
      sr[c] = __float_as_uint(fmaf(__uint_as_float(sr[c]) * st.f, k.x, e.x));
      sr[c + 1] = __float_as_uint(fmaf(__uint_as_float(sr[c + 1]) * st.f, k.y, e.y));
      sr[c + 2] = __float_as_uint(fmaf(__uint_as_float(sr[c + 2]) * st.f, k.z, e.z));
      sr[c + 3] = __float_as_uint(fmaf(__uint_as_float(sr[c + 3]) * st.f, k.w, e.w));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        sr[c + i] = __float_as_uint(__uint_as_float(sr[c + i]) * st.f);
    }
  }
  if (edge) {
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      const int pos = kb0 + c0 + c;
      const int j = pos - len;
      const bool see = j < 0 || (pos < end && (seen >> (j & 63) & 1));
      if (!see) sr[c] = __float_as_uint(-INFINITY);
    }
  }
  constexpr int kChains = CW < 8 ? CW : 8;
  float mp[kChains];
#pragma unroll
  for (int e = 0; e < kChains; ++e) mp[e] = __uint_as_float(sr[e]);
#pragma unroll
  for (int c = kChains; c < CW; c += kChains)
#pragma unroll
    for (int e = 0; e < kChains; ++e) mp[e] = fmaxf(mp[e], __uint_as_float(sr[c + e]));
  float mx = mp[0];
#pragma unroll
  for (int e = 1; e < kChains; ++e) mx = fmaxf(mx, mp[e]);
  mx -= Lazy<F8>::kPScaleLog2;
  const bool move = __any_sync(0xffffffffu, mx > st.m + Lazy<F8>::kLog2);
  float alpha = 1.0f;
  if (move) {
    const float m_new = fmaxf(st.m, mx);
    alpha = m_new == -INFINITY ? 1.0f : ex2_approx(st.m - m_new);
    st.l *= alpha;
    st.m = m_new;
  }
  const float m_use = st.m == -INFINITY ? 0.0f : st.m;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  // P, eight words at a time, over S's columns (all of them in registers)
  constexpr int kOwn = 32 / REP;  // words of P that hold this copy's keys
#pragma unroll
  for (int w0 = 0; w0 < kOwn; w0 += 8) {
    uint32_t hi[8], lo[F8 ? 8 : 1];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int w = w0 + i;
      if constexpr (F8) {
        float pr[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) pr[k] = ex2_approx(__uint_as_float(sr[4 * w + k]) - m_use);
        const float4 v = *reinterpret_cast<const float4*>(table + 256 + 4 * w);
        sum[0] = fmaf(pr[0], v.x, sum[0]);
        sum[1] = fmaf(pr[1], v.y, sum[1]);
        sum[2] = fmaf(pr[2], v.z, sum[2]);
        sum[3] = fmaf(pr[3], v.w, sum[3]);
        split4(pr[0], pr[1], pr[2], pr[3], hi[i], lo[i]);
      } else {
        const float p0 = ex2_approx(__uint_as_float(sr[2 * w]) - m_use);
        const float p1 = ex2_approx(__uint_as_float(sr[2 * w + 1]) - m_use);
        sum[i & 3] += p0 + p1;
        hi[i] = pack_bf16x2(p0, p1);
      }
    }
    const uint32_t col = tlane + kq * kOwn + w0;
    tmem_st8(col, hi);
    if constexpr (F8) tmem_st8(col + 32, lo);
  }
  st.l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
#pragma unroll
  for (int r = 0; r < REP; ++r)
    if (r != kq) {
#pragma unroll
      for (int w = 0; w < kOwn; w += 8) {
        tmem_st8_zero(tlane + r * kOwn + w);
        if constexpr (F8) tmem_st8_zero(tlane + 32 + r * kOwn + w);
      }
    }
  if (move && !first) {
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t r[32];
      tmem_ld32(tlane + kOCol + c * 32, r);
      tmem_ld_wait();
      reg_pin(r);
#pragma unroll
      for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
      tmem_st32(tlane + kOCol + c * 32, r);
    }
  }
  tmem_st_wait();
}

// ------------------------------------------------------------ the kernel
template <int D, bool F8, int REP>
__global__ void __launch_bounds__(kTreeThreads, 2)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ TreeParams p) {
  using L = TreeLayout<D, F8>;
  constexpr int KT = L::kTile;
  constexpr int kSt = L::kStages;
  constexpr int RS = kSoftThreads / REP;  // distinct query rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  TreeBars* bars = reinterpret_cast<TreeBars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int share = blockIdx.x / p.row_tiles;
  const int rt = blockIdx.x % p.row_tiles;

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_ready, kSoftThreads);
    for (int s = 0; s < kSt; ++s) {
      mbar_init(&bars->k_full[s], 1);
      mbar_init(&bars->k_empty[s], 1);
      mbar_init(&bars->v_full[s], 1);
      mbar_init(&bars->v_empty[s], 1);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      mbar_init(&bars->sc_full[s], 1);
      mbar_init(&bars->sc_empty[s], 4);
    }
    mbar_init(&bars->s_full, 1);
    mbar_init(&bars->p_ready, kSoftThreads);
    mbar_init(&bars->o_full, 1);
    mbar_init(&bars->drain, 1);
    bars->bad_lo = bars->bad_hi = 0;
    // an earlier CTA already recorded a pipeline timeout: exit without work
    bars->abort_flag = (*static_cast<volatile unsigned int*>(&g_tree_error) != 0) ? 1 : 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    // the share: tiles [x0, x0 + count) of the list of all pairs' tiles
    const int total = all_tiles(p, KT);
    const int size = share_size(total, p.shares);
    const long long x0 = static_cast<long long>(share) * size;
    const int count = static_cast<int>(min(max(total - x0, 0ll), static_cast<long long>(size)));
    if (lane == 0) {
      bars->count = count;
      bars->start_b = bars->start_h = bars->start_t = 0;
    }
    __syncwarp();
    if (count > 0) {
      int before = 0;  // tiles of the sequences before this batch of 32
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int n = b0 + lane < p.B ? seq_tiles(p, b0 + lane, KT) * p.Hkv : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const int lo = before + incl - n;
        if (n > 0 && x0 >= lo && x0 < lo + n) {
          const int off = static_cast<int>(x0) - lo, nt = n / p.Hkv;
          bars->start_b = b0 + lane;
          bars->start_h = off / nt;
          bars->start_t = off % nt;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
        if (x0 < before) break;
      }
    }
  }
  __syncthreads();
  if (bars->abort_flag || bars->count == 0) return;
  if (warp == kTreeMmaWarp) {
    tmem_alloc(&bars->tmem_base, kTreeTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t sQ = smem_u32(smem + L::kQ);
  const uint32_t sK = smem_u32(smem + L::kK);
  const uint32_t sV = smem_u32(smem + L::kV);

  if (warp == kTreeTmaWarp) {
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      tma_prefetch_desc(&tk);
      tma_prefetch_desc(&tv);
      int it = 0;
      bool ok = true;
      for (Walk w(bars); ok && w.valid(p, KT); w.next(p)) {
        const int bh = w.b * p.Hkv + w.h;
        for (int t = 0; t < w.n; ++t, ++it) {
          const int s = it % kSt;
          const uint32_t ph = (it / kSt) & 1;
          const int kb0 = (w.t0 + t) * KT;
          if (!(ok = t_wait(&bars->k_empty[s], ph ^ 1, bars, 0x501))) break;
          mbar_arrive_expect_tx(&bars->k_full[s], L::kKvBytes);
#pragma unroll
          for (int c = 0; c < static_cast<int>(L::kRow / L::kAtom); ++c)
            tma_load_3d(smem + L::kK + s * L::kKvBytes + c * (KT * L::kAtom), &tk,
                        &bars->k_full[s], c * 64, kb0, bh);
          if (F8) {
            const int ss = it % kScaleSlots;
            if (!(ok = t_wait(&bars->sc_empty[ss], ((it / kScaleSlots) & 1) ^ 1, bars, 0x502)))
              break;
            const uint32_t bytes = static_cast<uint32_t>(min(KT, p.cap - kb0));
            const long long at = static_cast<long long>(bh) * p.cap + kb0;
            mbar_arrive_expect_tx(&bars->sc_full[ss], 2 * bytes);
            bulk_load(smem + L::kScale + ss * 256, p.k_scale + at, bytes, &bars->sc_full[ss]);
            bulk_load(smem + L::kScale + ss * 256 + 128, p.v_scale + at, bytes,
                      &bars->sc_full[ss]);
          }
          if (!(ok = t_wait(&bars->v_empty[s], ph ^ 1, bars, 0x503))) break;
          mbar_arrive_expect_tx(&bars->v_full[s], L::kKvBytes);
#pragma unroll
          for (int c = 0; c < static_cast<int>(L::kRow / L::kAtom); ++c)
            tma_load_3d(smem + L::kV + s * L::kKvBytes + c * (KT * L::kAtom), &tv,
                        &bars->v_full[s], c * 64, kb0, bh);
        }
      }
    }
    __syncwarp();
  } else if (warp == kTreeMmaWarp) {
    // ------------------------------------------------ MMA issuer
    if (lane == 0) {
      int it = 0, seg = 0;
      bool ok = true;
      for (Walk w(bars); ok && w.valid(p, KT); w.next(p), ++seg) {
        if (!(ok = t_wait(&bars->q_ready, seg & 1, bars, 0x511))) break;
        for (int t = 0; t < w.n; ++t, ++it) {
          const int s = it % kSt;
          const uint32_t ph = (it / kSt) & 1;
          if (!(ok = t_wait(&bars->k_full[s], ph, bars, 0x512))) break;
          tc_fence_after_sync();
          const uint32_t kbase = sK + s * L::kKvBytes;
          if constexpr (F8) {
            constexpr uint32_t idesc_s = idesc_e4m3_f32(128, KT);
#pragma unroll
            for (int i = 0; i < 2 * (D / 32); ++i) {
              const int piece = i / (D / 32), kk = i % (D / 32);
              umma_ss_f8(tmem, sdesc<L::kAtom>(sQ + piece * L::kQChunk + kk * 32, 16, 8 * L::kAtom),
                         sdesc<L::kAtom>(kbase + kk * 32, 16, 8 * L::kAtom), idesc_s,
                         i > 0 ? 1u : 0u);
            }
          } else {
            constexpr uint32_t idesc_s = idesc_bf16_f32(128, KT, false, false);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              umma_ss(tmem, sdesc_sw128(sQ + (kk >> 2) * L::kQChunk + (kk & 3) * 32, 16, 1024),
                      sdesc_sw128(kbase + (kk >> 2) * (KT * 128) + (kk & 3) * 32, 16, 1024),
                      idesc_s, kk > 0 ? 1u : 0u);
          }
          umma_commit(&bars->k_empty[s]);
          umma_commit(&bars->s_full);  // also: PV of the tile before is complete
          if (!(ok = t_wait(&bars->p_ready, it & 1, bars, 0x513) &&
                     t_wait(&bars->v_full[s], ph, bars, 0x514)))
            break;
          tc_fence_after_sync();
          const uint32_t vbase = sV + s * L::kKvBytes;
          if constexpr (F8) {
            constexpr uint32_t idesc_pv = idesc_e4m3_f32(128, D) | (1u << 16);  // B MN-major
#pragma unroll
            for (int i = 0; i < 2 * (KT / 32); ++i) {
              const int piece = i / (KT / 32), kk = i % (KT / 32);
              umma_ts_f8(tmem + kOCol, tmem + piece * 32 + kk * 8,
                         sdesc<L::kAtom>(vbase + kk * 32 * L::kAtom, 16, 8 * L::kAtom), idesc_pv,
                         (t > 0 || i > 0) ? 1u : 0u);
            }
          } else {
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, false, true);
#pragma unroll
            for (int kk = 0; kk < KT / 16; ++kk)
              umma_ts(tmem + kOCol, tmem + kk * 8,
                      sdesc_sw128(vbase + kk * 2048, KT * 128, 1024), idesc_pv,
                      (t > 0 || kk > 0) ? 1u : 0u);
          }
          umma_commit(&bars->v_empty[s]);
          if (t == w.n - 1) umma_commit(&bars->o_full);
        }
      }
      umma_commit(&bars->drain);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax and epilogue
    // A failed wait clears ok: the warp then skips the work that is left, but
    // not the epilogue barriers, which the four warps pass together.
    const int tid = threadIdx.x;
    const int rs = tid % RS, kq = tid / RS;
    const uint32_t tlane = tmem_addr(tmem, warp * 32, 0);
    float* table = reinterpret_cast<float*>(smem + L::kTable) + warp * 384;
    int it = 0, seg = 0;
    bool ok = true;
    for (Walk w(bars); w.left > 0; w.next(p), ++seg) {
      if (tid == 0) {
        bars->pair_tiles = seq_tiles(p, w.b, KT);
        bars->pair_len = seq_len(p, w.b);
        bars->bad_lo = bars->bad_hi = 0;
      }
      named_bar_sync(1, kSoftThreads);
      w.set(bars->pair_tiles);
      const int len = bars->pair_len;
      const int r = rt * 128 + rs;
      const bool exists = r < p.R;
      const int end = min(len + p.T, p.cap);
      const long long row0 = (static_cast<long long>(w.b) * p.Hkv + w.h) * p.R;  // of o, lse
      RowState st;
      st.m = -INFINITY;
      st.l = 0.0f;
      const int eq = store_query<D, F8>(smem + L::kQ, p.q + (row0 + r) * (D / 8), exists, tid);
      st.f = F8 ? p.scale_log2 * pow2_of(eq) : p.scale_log2;
      fence_proxy_async_smem();
      mbar_arrive(&bars->q_ready);
      // mask row of this thread's draft, and the drafts that some row sees
      unsigned long long seen = 0, any = 0;
      if (p.mask) {
        const unsigned long long* mk = p.mask + w.b * p.mask_stride;
        if (exists) seen = __ldg(mk + r % p.T);
        if (lane < p.T) any = __ldg(mk + lane);
        if (lane + 32 < p.T) any |= __ldg(mk + lane + 32);
        any = static_cast<unsigned long long>(
                  __reduce_or_sync(0xffffffffu, static_cast<unsigned>(any >> 32)))
                  << 32 |
              __reduce_or_sync(0xffffffffu, static_cast<unsigned>(any));
      } else {
        seen = (2ull << (r % p.T)) - 1;
        any = (2ull << (p.T - 1)) - 1;
      }
      for (int t = 0; ok && t < w.n; ++t, ++it) {
        const int kb0 = (w.t0 + t) * KT;
        const bool edge = kb0 + KT > len;
        if (edge) {
          const int s = it % kSt;
          ok = __all_sync(0xffffffffu, t_wait(&bars->v_full[s], (it / kSt) & 1, bars, 0x521));
          if (!ok) break;
          clean_values<D, F8>(smem + L::kV + s * L::kKvBytes, kb0, len, end, any, bars);
          fence_proxy_async_smem();
        }
        if constexpr (F8) {
          // this warp's columns of the scale table; a byte behind the last row is
          // kept to finite powers (its P is zero)
          constexpr int CW = KT / REP;
          const int ss = it % kScaleSlots;
          ok = __all_sync(0xffffffffu, t_wait(&bars->sc_full[ss], (it / kScaleSlots) & 1, bars, 0x522));
          if (!ok) break;
          const uint8_t* raw = smem + L::kScale + ss * 256 + kq * CW;
          for (int c = lane; c < CW; c += 32) {
            const int e = min(max(static_cast<int>(raw[128 + c]), 1), 253) - 127;
            table[c] = __uint_as_float(static_cast<uint32_t>(raw[c]) << 23);
            table[128 + c] = static_cast<float>(e);
            table[256 + c] = pow2_of(-e);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->sc_empty[ss]);
        }
        ok = __all_sync(0xffffffffu, t_wait(&bars->s_full, it & 1, bars, 0x523));
        if (!ok) break;
        tc_fence_after_sync();
        softmax_tile<D, F8, REP>(tlane, kq, st, table, t == 0, edge, kb0, len, end, seen);
        tc_fence_before_sync();
        mbar_arrive(&bars->p_ready);
        if constexpr (F8) __syncwarp();  // the table is rewritten for the next tile
      }
      if (ok) ok = __all_sync(0xffffffffu, t_wait(&bars->o_full, seg & 1, bars, 0x524));
      tc_fence_after_sync();
      // ---- epilogue: merge the copies of a row, then o and lse or a partial
      bars->row_m[tid] = st.m;
      bars->row_l[tid] = st.l;
      named_bar_sync(1, kSoftThreads);
      float m_all = bars->row_m[rs];
#pragma unroll
      for (int i = 1; i < REP; ++i) m_all = fmaxf(m_all, bars->row_m[rs + i * RS]);
      const float m_ref = m_all == -INFINITY ? 0.0f : m_all;
      const float mine = ex2_approx(st.m - m_ref);  // 0 for a copy that saw nothing
      float l_all = 0.0f;
#pragma unroll
      for (int i = 0; i < REP; ++i) {
        const float li = bars->row_l[rs + i * RS];
        l_all += li == 0.0f ? 0.0f : li * ex2_approx(bars->row_m[rs + i * RS] - m_ref);
      }
      named_bar_sync(1, kSoftThreads);
      const bool whole = w.t0 == 0 && w.n == w.nt;
      const float inv = !whole ? 1.0f : (l_all == 0.0f ? 0.0f : 1.0f / l_all);
      if (kq == 0) bars->row_l[rs] = inv;
      // a share's first pair goes to slot 0, its last to slot 1
      const long long slot = 2ll * blockIdx.x + (seg == 0 ? 0 : 1);
      if (kq == 0 && exists && ok) {
        if (whole)
          p.lse[row0 + r] = l_all == 0.0f ? -INFINITY : (m_ref + log2f(l_all)) * kLn2;
        else
          p.part_ml[slot * p.prow + rs] = make_float2(m_all, l_all);
      }
      const unsigned long long bad =
          static_cast<unsigned long long>(bars->bad_hi) << 32 | bars->bad_lo;
      float4* buf = reinterpret_cast<float4*>(smem + L::kQ);  // row x 4 units, rotated by row
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 16) {
        uint32_t x[16];
        tmem_ld<16>(tlane + kOCol + c0, x);
        tmem_ld_wait();
        reg_pin(x);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          buf[tid * 4 + (u ^ ((tid >> 1) & 3))] =
              make_float4(__uint_as_float(x[4 * u]) * mine, __uint_as_float(x[4 * u + 1]) * mine,
                          __uint_as_float(x[4 * u + 2]) * mine,
                          __uint_as_float(x[4 * u + 3]) * mine);
        named_bar_sync(1, kSoftThreads);
#pragma unroll
        for (int i = 0; i < RS * 4 / kSoftThreads; ++i) {
          const int row = (tid >> 2) + i * (kSoftThreads / 4), u = tid & 3;
          const int rr = rt * 128 + row;
          if (rr < p.R && ok) {
            float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < REP; ++q) {
              const int ln = row + q * RS;
              const float4 z = buf[ln * 4 + (u ^ ((ln >> 1) & 3))];
              y[0] += z.x;
              y[1] += z.y;
              y[2] += z.z;
              y[3] += z.w;
            }
            const float f = bars->row_l[row];
            const int col = c0 + 4 * u;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] *= f;
            if (bad) {
              // drafts with NaN or infinities that this row sees
              unsigned long long hit =
                  bad & (p.mask ? __ldg(p.mask + w.b * p.mask_stride + rr % p.T)
                                : (2ull << (rr % p.T)) - 1);
              while (hit) {
                const int j = __ffsll(static_cast<long long>(hit)) - 1;
                hit &= hit - 1;
                const long long at =
                    (static_cast<long long>(w.b) * p.Hkv + w.h) * p.cap + len + j;
                for (int e = 0; e < 4; ++e) {
                  if (F8) {
                    if ((p.v[at * D + col + e] & 0x7f) == 0x7f) y[e] = NAN;
                  } else {
                    const float v = __bfloat162float(
                        reinterpret_cast<const __nv_bfloat16*>(p.v)[at * D + col + e]);
                    if (!isfinite(v)) y[e] += v;
                  }
                }
              }
            }
            if (whole)
              *reinterpret_cast<uint2*>(p.o + (row0 + rr) * D + col) =
                  make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
            else
              *reinterpret_cast<float4*>(p.part_o + (slot * p.prow + row) * D + col) =
                  make_float4(y[0], y[1], y[2], y[3]);
          }
        }
        named_bar_sync(1, kSoftThreads);
      }
    }
  }

  // ------------------------------------------------ teardown
  if (warp == kTreeMmaWarp) mbar_wait(&bars->drain, 0, &bars->abort_flag, &g_tree_error, 0x5ff);
  if (bars->abort_flag) {
    // let any bulk copy already in flight land before the CTA exits
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kTreeMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, kTreeTmemCols);
  }
}

// ------------------------------------------------------------ merge
// One block a query row: where several shares cover the row's pair, the row's
// partials are merged, four warps over the shares.
template <int D, int KT>
__global__ void __launch_bounds__(128) fa_tree_combine(const __grid_constant__ TreeParams p) {
  constexpr int kC = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = blockIdx.x;  // of o: ((b * Hkv + h) * R + r)
  const int r = static_cast<int>(row % p.R);
  const long long bh = row / p.R;
  const int b = static_cast<int>(bh / p.Hkv), h = static_cast<int>(bh % p.Hkv);
  int total = 0, before = 0;
  for (int i = lane; i < p.B; i += 32) {
    const int n = seq_tiles(p, i, KT);
    total += n;
    if (i < b) before += n;
  }
  total = warp_sum(total) * p.Hkv;
  const int nt = seq_tiles(p, b, KT);
  const int s0 = warp_sum(before) * p.Hkv + h * nt;
  const int size = share_size(total, p.shares);
  const int first = s0 / size, last = (s0 + nt - 1) / size;
  if (first == last) return;
  const int rt = r / 128, rs = r % 128;
  __shared__ float sm[4], sl[4], so[4][D];
  float m = -INFINITY;
  for (int c = first + lane; c <= last; c += 32) {
    // the pair is the share's first unless it starts inside the share
    const long long slot = 2ll * (static_cast<long long>(c) * p.row_tiles + rt) +
                           (c == first && s0 != c * size ? 1 : 0);
    m = fmaxf(m, p.part_ml[slot * p.prow + rs].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float m_ref = m == -INFINITY ? 0.0f : m;
  float l = 0.0f, acc[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) acc[c] = 0.0f;
  for (int c = first + warp; c <= last; c += 4) {
    const long long slot = 2ll * (static_cast<long long>(c) * p.row_tiles + rt) +
                           (c == first && s0 != c * size ? 1 : 0);
    const float2 ml = p.part_ml[slot * p.prow + rs];
    if (ml.y == 0.0f) continue;  // this share's keys are all unseen
    const float wgt = ex2_approx(ml.x - m_ref);
    l = fmaf(wgt, ml.y, l);
    const float* src = p.part_o + (slot * p.prow + rs) * D + lane * kC;
#pragma unroll
    for (int k = 0; k < kC; ++k) acc[k] = fmaf(wgt, src[k], acc[k]);
  }
#pragma unroll
  for (int k = 0; k < kC; ++k) so[warp][lane * kC + k] = acc[k];
  if (lane == 0) {
    sm[warp] = m_ref;
    sl[warp] = l;
  }
  __syncthreads();
  const float l_all = (sl[0] + sl[1]) + (sl[2] + sl[3]);
  const float inv = l_all == 0.0f ? 0.0f : 1.0f / l_all;
  if (threadIdx.x < D)
    p.o[row * D + threadIdx.x] =
        __float2bfloat16_rn(((so[0][threadIdx.x] + so[1][threadIdx.x]) +
                             (so[2][threadIdx.x] + so[3][threadIdx.x])) * inv);
  if (threadIdx.x == 0)
    p.lse[row] = l_all == 0.0f ? -INFINITY : (m_ref + log2f(l_all)) * kLn2;
}

template <int D, bool F8, int REP>
cudaError_t launch_tile(const TreeParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t s) {
  constexpr uint32_t smem = TreeLayout<D, F8>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(fa_tree_kernel<D, F8, REP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  fa_tree_kernel<D, F8, REP>
      <<<static_cast<unsigned>(p.shares) * p.row_tiles, kTreeThreads, smem, s>>>(tk, tv, p);
  return cudaGetLastError();
}

template <int D, bool F8>
cudaError_t launch_type(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t s) {
  const TreePlan plan = tree_plan(a.c, a.Hq, a.T, 2 * a.num_sms);
  TreeParams p{};
  p.q = static_cast<const uint4*>(a.q);
  p.lens = a.lens;
  p.mask = a.mask;
  p.mask_stride = a.mask_stride;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.B = a.c.B;
  p.Hkv = a.c.Hkv;
  p.cap = a.c.cap;
  p.G = a.Hq / a.c.Hkv;
  p.T = a.T;
  p.R = p.G * a.T;
  p.row_tiles = plan.row_tiles;
  p.shares = plan.shares;
  p.prow = plan.prow;
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + static_cast<size_t>(plan.slots) * plan.prow * D);
  p.k_scale = a.c.k_scale;
  p.v_scale = a.c.v_scale;
  p.v = static_cast<const uint8_t*>(a.c.v);
  p.scale_log2 = a.scale * kLog2e;
  const cudaError_t e = p.R <= 32   ? launch_tile<D, F8, 4>(p, tk, tv, s)
                        : p.R <= 64 ? launch_tile<D, F8, 2>(p, tk, tv, s)
                                    : launch_tile<D, F8, 1>(p, tk, tv, s);
  if (e != cudaSuccess || plan.slots == 0) return e;
  const long long rows = static_cast<long long>(p.B) * a.Hq * a.T;
  fa_tree_combine<D, TreeLayout<D, F8>::kTile><<<static_cast<unsigned>(rows), 128, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decode_tree(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                               cudaStream_t s) {
  if (a.c.format == FA_CACHE_E4M3)
    return a.c.d == 64 ? launch_type<64, true>(a, tk, tv, s) : launch_type<128, true>(a, tk, tv, s);
  return a.c.d == 64 ? launch_type<64, false>(a, tk, tv, s) : launch_type<128, false>(a, tk, tv, s);
}

cudaError_t tree_read_clear_error(uint32_t* out, cudaStream_t s) {
  cudaError_t e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  uint32_t v = 0;
  e = cudaMemcpyFromSymbol(&v, g_tree_error, sizeof(v));
  if (e != cudaSuccess) return e;
  if (v) {
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbol(g_tree_error, &zero, sizeof(zero));
  }
  *out = v;
  return e;
}

}  // namespace fa
