// fa_tree.cu — attention of a tree of drafted tokens over the key/value cache
// (bf16 or e4m3), grouped heads, a length for each sequence.
//
// The G = Hq / Hkv query heads of a key head times the T drafts are R = G T
// query rows against one key/value sequence: o = softmax(scale q k^T) v over the
// committed tokens and the drafts that the row's mask names.  Every key and
// value is read once a row tile, and ~4 R FLOPs are done for each of its
// elements: HBM's time is the floor up to a hundred rows, and it is reached for the few
// rows of a decode step over long caches.  The products run on the tensor core for all.
//
// Split.  The (sequence, key head) pairs are cut into tiles of 128 keys; a pair
// counts as many units as it has tiles and kPairCost for its start and end, and
// the list of all units is cut into equal shares, one CTA a share (times the row
// tiles of 64 rows, which run side by side so that they read a key tile while it
// is in L2).  Lengths live on the device, so each CTA finds its share from lens
// itself.  A pair that one CTA covers is finished there; the partial results of
// the others (o and its log-sum-exp, at most two a CTA) go to the workspace, and
// fa_tree_combine merges them by the running-maximum update.
//
// Products.  The keys take the tensor core's 128 rows and the query rows its
// columns: S^T = K Q^T (M = 128 keys, N = NR query rows, 16, 32 or 64) and
// O^T = V^T P^T (M = d channels, N = NR).  With the query rows as M, a decode
// step's 1-64 rows would be padded to 128 and every tile would pay for them:
// 1024 cycles a tile of e4m3, measured 3900 with the softmax between, against
// 1434 that HBM gives.  This way a tile costs 512 or less, one thread owns one key
// (its scale, its visibility), and any R keeps all four softmax warps busy.
//
// One CTA (two an SM up to 32 rows, one for 64):
//   * one warp streams K and V tiles through one TMA ring, in the order the
//     tensor core takes them: K0 K1 V0 K2 V1 ...;
//   * one (two where the CTA has the SM alone) issues S^T(t + 2) once softmax(t) has
//     read the buffer before it, and PV(t): S^T has two buffers in tensor memory;
//   * four warps for every 16 rows, a key a thread: softmax over the columns, P^T to shared
//     memory ([key][row], an operand as it lies), epilogue with a channel a thread.
//     Four warps share a row's reference M; one barrier a tile tells them whether
//     some score of their 16 rows passed it by more than Lazy binades, and only then
//     maxima are exchanged and O is rescaled.  The next pair's queries are stored
//     during a pair's last tile, so that its first scores are ready when the
//     epilogue ends.
//
// e4m3 operands: kind::f8f6f4 takes the cache as it lies in memory.  Two e4m3
// pieces of 4 significant bits hold the 8 bits of a bf16 query exactly (its row
// scaled by a power of two into 448).  A probability is three e5m2 pieces of 3 bits,
// 2^-9 of it, over the 30 binades of that type: two e4m3 pieces have the bits but 15
// binades, and a long tail of small weights behind a heavy key was lost with them.  S
// accumulates both pieces of q; those of P are columns side by side, so that V is read
// once.  The scales of
// keys and values join in the softmax: with e_j the exponent of value row j and s_j =
// scale log2(e) 2^(k_j) S_j, a row keeps M = max (s_j + e_j); the sum takes
// p_j = 2^(s_j - M) and the product with the codes P_j = 2^(e_j) p_j, so that
// o = O / l needs no further factor.  A value row of zeros has the least e_j there is:
// its p_j may be far above 1, and is not lost however large the other rows are.
//
// Measured (d = 128, 8 key heads, the cache larger than L2; % of the rate of a plain
// copy, 6.79 TB/s): 8 rows over 8 sequences of 32K keys 88 us in e4m3 (90 %; 113 us
// and 71 % for 64K keys of d = 64) and 163 us in bf16 (97 %): HBM.  64 rows over 4 sequences
// of 32K to 64K keys in bf16 127 us (92 %), in e4m3 120 us (49 %): the softmax, 16 warps
// that issue half of the cycles (2000 a tile of 128 keys by 64 rows), with long waits for
// tensor memory and the group barrier.  256 rows over 8 sequences of 4K to 8K keys in bf16
// 91 us: shared memory, whose 176 KB a tile of 64 rows take 1375 of its 1400 cycles, and
// starts and ends of pairs (5 us each).  32 rows over 32 sequences of 500 to 4096 keys in e4m3 47 us (49 %): starts
// and ends of pairs, the first loads (5 us) and the merge (5 us).  One token over 1000
// keys 13.5 us.  Over 64 rows an e4m3 cache is slower than one in bf16: 128 rows over 8
// sequences of 32K keys 279 us against 205, the 256 rows above 123 us, since every tile
// of 64 rows splits all its probabilities into pieces.
#include <atomic>
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

constexpr int kTile = kTreeTile;  // keys a tile: one a softmax thread
constexpr int kMaxSlots = 8;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

constexpr int kPairCost = kTreePairCost;

constexpr int kNoExponent = 1000;  // of rows of zeros

// -M of a row that has seen no key: any finite score passes the reference, and
// -inf stays -inf.
constexpr float kUnseen = 1e38f;

// e4m3 queries: the pieces of a row tile's queries share one power of two, 2^e of the
// tile's largest element, where each row's own would be at most 2^kNear smaller; a
// product of an element and a code is then off by at most 2^-12.8 of the row's largest.  Rows
// that differ by more (a padded row may hold anything) have each its own power of two
// and the softmax a product more for two scores, through local memory: 64 rows over 4 x 8
// heads of 32K to 64K keys take 183 instead of 117 us so.
struct Queries {
  static constexpr int kNear = 4;
  static constexpr float kByRow = -1.0f;  // in place of the factor of all rows
};

// A row's accumulator is rescaled only when its maximum grows by more than
// kLog2 binades.  bf16 has the range for any P; for e4m3 P is scaled so that 2^kLog2
// times the largest P at the last rescale is 2^15, about as much as fp16 holds.
template <bool F8>
struct Lazy {
  static constexpr float kLog2 = F8 ? 6.0f : 8.0f;
  static constexpr float kTop = F8 ? 15.0f : 8.0f;             // log2 of the largest P
  [[maybe_unused]] static constexpr float kLowScale = 0.125f;  // unit of the lower pieces
  // Value rows of smaller exponents enter M with this one: their p = 2^(s - M) is at most
  // 2^(kTop + 82), and a sum over 2^28 keys stays below 2^126 (as 1 / l is formed).
  [[maybe_unused]] static constexpr float kLeastExponent = -82.0f;
};

// A pair of the share: its tiles t0 .. t0 + tiles - 1 are worked on here.
struct PairInfo {
  long long bh;
  int b, h, u0, len, nt, t0, tiles;
  int valid;               // 0 behind the last pair
  unsigned int bad[2];     // drafts whose value row holds NaN or infinities
  unsigned long long any;  // drafts that some row of the sequence sees
  int qmax, qmin;          // e4m3: greatest and least exponent of the tile's queries
};

struct TreeBars {
  uint64_t q_ready;
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t s_full[2], p_ready[2], pv_done[2], drain;  // by tile parity
  uint32_t tmem_base;
  int abort_flag;
  int start_b, start_h, start_u0, unit0, unit1;  // this CTA's share
  int lens[32];                                  // lengths of sequences start_b, start_b + 1, ...
  PairInfo pair[4];                              // by pair, as the softmax warps agree on them
};

// What the softmax threads know of a pair's query rows.
template <int NR>
struct TreeRows {
  unsigned long long seen[NR];  // mask row
  float m[NR];      // reference exponent, -inf before the first key
  float neg_m[NR];  // its negative: kUnseen before the first key, -inf for rows past R
  float unit[NR];   // scale log2(e) times the unit of the row's query pieces (see Queries)
  float alpha[NR];  // of the last move, its square root
  float inv[NR];    // epilogue: what O is multiplied by
  float part[4][NR];            // a warp's maximum or sum
};

// Address of 16-byte unit c of row r in a tile of ATOM-byte rows, swizzled over the
// row (128, 64 or 32 bytes).
template <uint32_t ATOM>
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t c) {
  constexpr uint32_t kUnits = ATOM / 16;
  return r * ATOM + (c ^ (r / (8 / kUnits) % kUnits)) * 16u;
}

template <int D, bool F8, int NR>
struct TreeLayout {
  static constexpr uint32_t kRow = F8 ? D : 2 * D;             // bytes of a cache row
  static constexpr uint32_t kAtom = F8 && D == 64 ? 64 : 128;  // swizzle width in bytes
  static constexpr int kBoxes = kRow / kAtom;                  // boxes of columns in a row
  // A tile comes in kParts slots: 64 columns of K, 64 keys of V (bf16, d = 128, where
  // two CTAs share the SM).
  static constexpr int kParts = tree_v_keys(!F8, D, NR) == kTile ? 1 : 2;
  static constexpr uint32_t kSlot = kTile * kRow / kParts;     // 16 KB or 8 KB
  static constexpr int kVKeys = kTile / kParts;
  static constexpr int kGroups = NR / 16;  // softmax: 128 threads (a key each) for 16 rows
  static constexpr int kSoft = kTile * kGroups;
  // With one CTA an SM the two products have an issuing warp each: one warp's 16
  // instructions and their waits took 2000 cycles a tile, more than the softmax.
  static constexpr int kMmaWarps = tree_ctas(NR) == 1 ? 2 : 1;
  static constexpr int kTmaWarp = kSoft / 32, kMmaWarp = kTmaWarp + 1;  // and the S warp behind
  static constexpr int kThreads = kSoft + 32 + 32 * kMmaWarps;
  static constexpr int kPieces = F8 ? 2 : 1;                   // of q
  static constexpr uint32_t kQPiece = NR * kRow;               // 64 columns at a time for bf16
  // P lies as [key][row], for e4m3 its three pieces one behind the other in a key's row of
  // 64 or 128 bytes (or two of 128 in boxes kPBox apart); the rest of the row is not used.
  static constexpr int kPPieces = F8 ? 3 : 1;
  static constexpr uint32_t kPAtom = F8 ? (NR == 16 ? 64 : 128) : 2 * NR;  // swizzle width
  static constexpr uint32_t kPBox = kTile * kPAtom;
  static constexpr uint32_t kPBytes = F8 && NR == 64 ? 2 * kPBox : kPBox;
  // 16-byte unit u of a key's P
  static __device__ __forceinline__ uint32_t p_at(int key, int u) {
    constexpr int kUnits = kPAtom / 16;
    return u / kUnits * kPBox + swizzled<kPAtom>(key, u % kUnits);
  }
  static constexpr int kCtas = tree_ctas(NR);                  // an SM
  static constexpr uint32_t kRoom = (kCtas == 2 ? 113u : 227u) * 1024 - 1024 - 1024 -
                                    2 * sizeof(TreeRows<NR>) - kPieces * kQPiece - 2 * kPBytes;
  static constexpr int kFit = kRoom / kSlot;
  // an even number, so that K and V tiles (K0 K1 V0 K2 V1 ...) each keep to their own
  // slots and a warp that waits for one of them knows the load before it complete
  static constexpr int kSlots = (kFit < kMaxSlots ? kFit : kMaxSlots) / 2 * 2;
  static_assert(kSlots >= 2 * kParts, "K(t + 1) is loaded before V(t)");
  static constexpr uint32_t kRing = 0;
  static constexpr uint32_t kQ = kRing + kSlots * kSlot;
  static constexpr uint32_t kP = kQ + kPieces * kQPiece;
  static constexpr uint32_t kRows = kP + 2 * kPBytes;
  static constexpr uint32_t kBar = kRows + 2 * sizeof(TreeRows<NR>);
  static constexpr uint32_t kUsed = kBar + 1024 + 1024;  // + alignment slack
  static_assert(kQ % 1024 == 0 && kP % 1024 == 0 && kRows % 16 == 0 && kBar % 8 == 0, "aligned");
  static constexpr uint32_t kSmem = kUsed > 81920u ? kUsed : 81920u;  // never three CTAs
  static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "fits");
  // tensor memory: S^T twice, O^T (of each piece)
  static constexpr uint32_t kOCol = 2 * NR;
  static constexpr uint32_t kOCols = kPPieces * NR;
  static constexpr uint32_t kCols = (F8 ? 8 : 4) * NR;
  static_assert(kOCol + kOCols <= kCols, "columns");
};
static_assert(sizeof(TreeBars) <= 1024, "barrier block");

struct TreeParams {
  const uint4* q;
  const int* lens;
  const unsigned long long* mask;
  long long mask_stride;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;     // [slots][prow][D]
  float* part_lse;   // [slots][prow], in units of ln 2
  int4* split;       // [shares], or null: see fa_tree_combine
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const uint8_t* v;  // the value cache, for rows with NaN or infinities
  int B, Hkv, cap, T, R;
  int row_tiles, shares, prow;
  float scale_log2;
};

// The bounded wait; its loop is out of line, so that a wait costs the kernel's
// hot code a few instructions (with the loops and other rare paths inlined the
// code was 100 KB, and warps waited for instructions a quarter of the time).
__device__ __noinline__ bool t_wait_loop(uint64_t* bar, uint32_t parity, TreeBars* b,
                                         uint32_t code) {
  return mbar_wait(bar, parity, &b->abort_flag, &g_tree_error, code);
}
__device__ __forceinline__ bool t_wait(uint64_t* bar, uint32_t parity, TreeBars* b, uint32_t code) {
  return mbar_try_wait(smem_u32(bar), parity) || t_wait_loop(bar, parity, b, code);
}

// The same wait by a whole warp, with one answer.
__device__ __forceinline__ bool all_wait(uint64_t* bar, uint32_t parity, TreeBars* b, uint32_t code) {
  return __all_sync(0xffffffffu, t_wait(bar, parity, b, code));
}

// One lane of a converged warp (the same one each time).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Keys of sequence b that exist: its committed tokens and its drafts.
__device__ __forceinline__ int seq_len(const TreeParams& p, int b) {
  return min(max(__ldg(p.lens + b), 0), p.cap);
}
__device__ __forceinline__ int seq_tiles(const TreeParams& p, int b) {
  return (min(seq_len(p, b) + p.T, p.cap) + kTile - 1) / kTile;
}

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The same through the share's first 32 lengths (a load behind the streams of all
// SMs takes 2 to 3 us).
__device__ __forceinline__ int near_len(const TreeParams& p, const TreeBars* bars, int b) {
  const int i = b - bars->start_b;
  return i < 32 ? bars->lens[i] : seq_len(p, b);
}
__device__ __forceinline__ int len_tiles(const TreeParams& p, int len) {
  return (min(len + p.T, p.cap) + kTile - 1) / kTile;
}

// Units of all (sequence, key head) pairs; the whole warp calls it.
__device__ __forceinline__ int all_units(const TreeParams& p) {
  int n = 0;
  for (int b = threadIdx.x & 31; b < p.B; b += 32) n += seq_tiles(p, b) + kPairCost;
  return warp_sum(n) * p.Hkv;
}

// Units a share: all shares but the last have this many.
__device__ __forceinline__ int share_size(int units, int shares) {
  return (units + shares - 1) / shares;
}

// A CTA's walk over the pairs whose tiles its share holds.  Pair (b, h) begins
// at unit u0, its tiles at u0 + kPairCost.
struct Walk {
  int b, h, u0, unit0, unit1;
  int t0, n, nt;  // first tile here, tiles here, tiles of the pair
  __device__ __forceinline__ explicit Walk(const TreeBars* bars)
      : b(bars->start_b), h(bars->start_h), u0(bars->start_u0), unit0(bars->unit0),
        unit1(bars->unit1), t0(0), n(0), nt(0) {}
  // Can the pair have tiles here?  (True for the first pair of a share with any.)
  __device__ __forceinline__ bool inside() const { return u0 + kPairCost < unit1; }
  __device__ __forceinline__ void set(int tiles) {
    nt = tiles;
    t0 = max(unit0 - u0 - kPairCost, 0);
    n = min(nt, unit1 - u0 - kPairCost) - t0;
  }
  __device__ __forceinline__ bool valid(const TreeParams& p, const TreeBars* bars) {
    if (!inside()) return false;
    set(len_tiles(p, near_len(p, bars, b)));
    return true;
  }
  __device__ __forceinline__ void next(const TreeParams& p) {
    u0 += nt + kPairCost;
    if (++h == p.Hkv) {
      h = 0;
      ++b;
    }
  }
};

// The pair behind pair `from` (one thread).
__device__ __forceinline__ void next_pair(const TreeParams& p, TreeBars* bars, const PairInfo& from,
                                          PairInfo& to) {
  to.u0 = from.u0 + from.nt + kPairCost;
  to.valid = to.u0 + kPairCost < bars->unit1;
  if (!to.valid) return;
  to.h = from.h + 1;
  to.b = from.b;
  to.len = from.len;
  if (to.h == p.Hkv) {
    to.h = 0;
    ++to.b;
    to.len = near_len(p, bars, to.b);
  }
  to.bh = static_cast<long long>(to.b) * p.Hkv + to.h;
  to.nt = len_tiles(p, to.len);
  to.t0 = 0;
  to.tiles = min(to.nt, bars->unit1 - to.u0 - kPairCost);
  to.bad[0] = to.bad[1] = 0;
  to.qmax = -kNoExponent;
  to.qmin = kNoExponent;
}

// ------------------------------------------------------------ tensor memory
// 32 lanes x 16 columns, thread t of the warp gets lane (its warp's base + t).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr)
               : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// ------------------------------------------------------------ conversions
// Four fp32 P of 0 .. 2^15 as three e5m2 pieces each: a word of high pieces, and words of
// middle and low pieces times 2^3 (each has accumulator columns of its own).  e5m2 is
// the high byte of fp16, so that the high piece is P in fp16 cut to 3 significant bits,
// the rest of it, exact in fp16 and below 2^-2 of P's binade, is cut the same way, and
// what then remains is rounded (half up): 2^-9 of P together, and 2^-20 where the last
// two are subnormal.  With a row's largest P at 2^9 or more that is 2^-29 of it, and a
// sum over 2^20 keys still within 2^-9.  Masks, additions and byte permutes run at four
// times the rate of the conversions to 8 bits.
__device__ __forceinline__ void split2(float x0, float x1, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  const uint32_t c = hi & 0xff00ff00u;
  const __half2 r = __hmul2(__hsub2(h, *reinterpret_cast<const __half2*>(&c)),
                            __half2half2(__ushort_as_half(0x4800)));  // 2^3
  mid = *reinterpret_cast<const uint32_t*>(&r);
  const uint32_t d = mid & 0xff00ff00u;
  const __half2 z = __hsub2(r, *reinterpret_cast<const __half2*>(&d));
  lo = *reinterpret_cast<const uint32_t*>(&z) + 0x00800080u;
}
__device__ __forceinline__ void split4(float x0, float x1, float x2, float x3, uint32_t& hi,
                                       uint32_t& mid, uint32_t& lo) {
  uint32_t h0, m0, l0, h1, m1, l1;
  split2(x0, x1, h0, m0, l0);
  split2(x2, x3, h1, m1, l1);
  hi = __byte_perm(h0, h1, 0x7531);
  mid = __byte_perm(m0, m1, 0x7531);
  lo = __byte_perm(l0, l1, 0x7531);
}

// Two fp32 of at most 448 as two e4m3 pieces each: hi = e4m3(x), lo = e4m3(x - hi).
// The subtraction is exact in fp16, and x has at most 8 bits here (a query).
__device__ __forceinline__ void split2_query(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const __nv_fp8x2_storage_t a =
      __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(h), __NV_SATFINITE, __NV_E4M3);
  const __half2 back = __half2(__nv_cvt_fp8x2_to_halfraw2(a, __NV_E4M3));
  hi = a;
  lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(h, back)), __NV_SATFINITE,
                                  __NV_E4M3);
}

__device__ __forceinline__ uint32_t word(const uint4& x, int k) {
  return k == 0 ? x.x : k == 1 ? x.y : k == 2 ? x.z : x.w;
}

// ------------------------------------------------------------ pairs of fp32
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// sdesc_sw128 with the swizzle of ATOM-byte rows.
template <uint32_t ATOM>
__device__ __forceinline__ uint64_t sdesc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  constexpr uint64_t kLayout = ATOM == 128 ? 2 : ATOM == 64 ? 4 : 6;
  return (sdesc_sw128(addr, lbo, sbo) & ~(7ull << 61)) | (kLayout << 61);
}

// ------------------------------------------------------------ query rows
// What a softmax thread reads of a pair besides keys and values.  It is asked for, into
// L2, a pair ahead, and loaded while the last product of the pair before runs.
template <int D, int NR>
struct PairLoads {
  static constexpr int kPer = kTile * (NR / 16) / NR;  // threads a query row
  static constexpr int kGran = D / 8 / kPer;           // eight channels each
  uint4 q[kGran];
  unsigned long long seen, any;  // mask rows: of row threadIdx.x, of drafts lane and lane + 32

  // trow: the draft of row threadIdx.x
  __device__ __forceinline__ void load(const TreeParams& p, int b, long long bh, int rt, int have,
                                       int trow) {
    const int r = threadIdx.x / kPer, part = threadIdx.x % kPer;
    const uint4* src = p.q + ((bh * p.R + rt * kTreeRows + r) * (D / 8) + part * kGran);
    const bool exists = r < have;
#pragma unroll
    for (int i = 0; i < kGran; ++i) q[i] = exists ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
    const int lane = threadIdx.x & 31;
    seen = (2ull << trow) - 1;
    any = 0;
    if (p.mask) {
      const unsigned long long* mk = p.mask + b * p.mask_stride;
      seen = __ldg(mk + trow);
      if (lane < p.T) any = __ldg(mk + lane);
      if (lane + 32 < p.T) any |= __ldg(mk + lane + 32);
    }
  }
  static __device__ __forceinline__ void ask(const TreeParams& p, int b, long long bh, int rt,
                                             int have, int trow) {
    const int r = threadIdx.x / kPer, part = threadIdx.x % kPer;
    if (r < have)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          p.q + ((bh * p.R + rt * kTreeRows + r) * (D / 8) + part * kGran)));
    if (p.mask && threadIdx.x < NR)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.mask + b * p.mask_stride + trow));
  }
  // The drafts that some row of the sequence sees.
  __device__ __forceinline__ unsigned long long drafts(const TreeParams& p) const {
    if (!p.mask) return (2ull << (p.T - 1)) - 1;
    return static_cast<unsigned long long>(
               __reduce_or_sync(0xffffffffu, static_cast<unsigned>(any >> 32)))
               << 32 |
           __reduce_or_sync(0xffffffffu, static_cast<unsigned>(any));
  }
};

// The row tile's query rows as the swizzled operand of S^T (rows past `have` are
// zeros), and their mask rows.  e4m3: two pieces of the rows times 2^-e (Queries).  The
// return value is scale log2(e), times 2^e, or kByRow.
template <int D, bool F8, int NR>
__device__ __forceinline__ float store_queries(uint8_t* sq, TreeRows<NR>* rows,
                                               const PairLoads<D, NR>& in, int have,
                                               float scale_log2, PairInfo* pair) {
  using L = TreeLayout<D, F8, NR>;
  constexpr int kPer = PairLoads<D, NR>::kPer, kGran = PairLoads<D, NR>::kGran;
  const int r = threadIdx.x / kPer, part = threadIdx.x % kPer;
  float factor = scale_log2;
  // a NaN or an infinity makes all scores of its row NaN, those too that would be -inf
  uint32_t all = 0;
#pragma unroll
  for (int i = 0; i < kGran; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) all = __vmaxu2(all, word(in.q[i], k) & 0x7fff7fffu);
  const uint32_t bad = __ballot_sync(0xffffffffu, max(all & 0xffffu, all >> 16) >= 0x7f80u);
  if (part == 0) {
    const bool nan = bad >> (threadIdx.x & 31) & ((1u << kPer) - 1);
    rows->m[r] = -INFINITY;
    rows->neg_m[r] = r >= have ? -INFINITY : nan ? NAN : kUnseen;
  }
  if (threadIdx.x < NR) rows->seen[threadIdx.x] = in.seen;
  if constexpr (!F8) {
#pragma unroll
    for (int i = 0; i < kGran; ++i) {
      const int c = part * kGran + i;  // 16-byte unit of the row
      *reinterpret_cast<uint4*>(sq + (c >> 3) * (NR * 128) + swizzled<128>(r, c & 7)) = in.q[i];
    }
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kGran; ++i) m = __vmaxu2(m, finite_max8(in.q[i]));
#pragma unroll
    for (int o = kPer / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m & 0xffffu, m >> 16);
    int e = scale_exponent(m);
    const int e_max = __reduce_max_sync(0xffffffffu, m ? e : -kNoExponent);
    const int e_min = __reduce_min_sync(0xffffffffu, m ? e : kNoExponent);
    if ((threadIdx.x & 31) == 0) {
      atomicMax(&pair->qmax, e_max);
      atomicMin(&pair->qmin, e_min);
    }
    named_bar_sync(1, L::kSoft);
    const int top = *static_cast<volatile int*>(&pair->qmax);
    if (top - *static_cast<volatile int*>(&pair->qmin) <= Queries::kNear) {
      e = top == -kNoExponent ? 0 : top;
      factor *= pow2_of(e);
    } else {
      if (part == 0) rows->unit[r] = scale_log2 * pow2_of(e);
      factor = Queries::kByRow;
    }
    const float s = pow2_of(-e);
#pragma unroll
    for (int i = 0; i < kGran; ++i) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        split2_query(bf_lo(word(in.q[i], k)) * s, bf_hi(word(in.q[i], k)) * s, hi[k], lo[k]);
      const int c = part * kGran + i;  // 8-byte half of a unit
      uint8_t* at = sq + swizzled<L::kAtom>(r, c >> 1) + (c & 1) * 8;
      *reinterpret_cast<uint2*>(at) = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
      *reinterpret_cast<uint2*>(at + L::kQPiece) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
    }
  }
  return factor;
}

// ------------------------------------------------------------ value rows
// A tile that reaches past the committed tokens: value rows that no query row
// of the sequence sees become zero (P is zero there, but 0 * NaN is not), and
// in drafts that some row sees NaN and infinities become zero and the draft is
// noted: the epilogue adds them to the rows that see it.  Key a thread and group of
// softmax warps: each group takes its part of the 16-byte units of the key's row sv,
// which is COLS boxes of ATOM bytes `stride` apart.  Neighbouring keys take the units
// in another order: in the same one, their rows' units lie in the same banks (6000
// cycles for a tile of 64 drafts in bf16 on one group).
template <uint32_t ATOM, int COLS, int GROUPS, bool F8>
__device__ __noinline__ void clean_values(uint8_t* sv, uint32_t stride, int key, int group, int pos,
                                          int len, int end, unsigned long long any,
                                          unsigned int* note) {
  constexpr int kBox = ATOM / 16, kUnits = COLS * kBox / GROUPS;  // of a box, of a group
  static_assert(kUnits * GROUPS == COLS * kBox, "units");
  if (pos < len) return;
  const int j = pos - len;
  const bool live = pos < end && (any >> (j & 63) & 1);
  const int order = key / (8 / kBox) % kBox;
  bool bad = false;
#pragma unroll 2
  for (int i = group * kUnits; i < (group + 1) * kUnits; ++i) {
    uint4* at = reinterpret_cast<uint4*>(sv + i / kBox * stride) + (i % kBox ^ order);
    if (!live) {
      *at = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4 x = *at;
    uint32_t w[4] = {x.x, x.y, x.z, x.w}, hit = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t n = F8 ? __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu)
                            : __vcmpgeu2(w[k] & 0x7fff7fffu, 0x7f807f80u);
      hit |= n;
      w[k] &= ~n;
    }
    if (hit) {
      *at = make_uint4(w[0], w[1], w[2], w[3]);
      bad = true;
    }
  }
  if (bad) atomicOr(note + (j >> 5 & 1), 1u << (j & 31));
}

// ------------------------------------------------------------ across lanes
// The sums of x[16] over the lanes: that of row l % 16 in lane l.  Each step
// halves the rows a lane holds.
__device__ __forceinline__ float sum_lanes(float (&x)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 8; n > 0; n >>= 1) {  // rows that a lane keeps
    const bool up = (lane & n) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? x[i] : x[i + n];
      const float keep = up ? x[i + n] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, n);
    }
  }
  return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 16);
}

// x = s - M of a key for 16 rows, or s + ev (where M is false), s = ks S; ks: scale
// log2(e), times 2^k and the unit of the query pieces for e4m3.
template <bool M>
__device__ __forceinline__ void form_scores(uint32_t taddr, const float* neg_m, float ks, float ev,
                                            f32x2 (&x)[8]) {
  uint32_t s[16];
  tmem_ld16(taddr, s);
  tmem_ld_wait();
  reg_pin(s);
  const f32x2 ks2 = pack2(ks, ks), ev2 = pack2(ev, ev);
#pragma unroll
  for (int r = 0; r < 8; r += 2) {
    ulonglong2 m = make_ulonglong2(ev2, ev2);
    if (M) m = *reinterpret_cast<const ulonglong2*>(neg_m + 2 * r);
    x[r] = fma2(pack2(__uint_as_float(s[2 * r]), __uint_as_float(s[2 * r + 1])), ks2, m.x);
    x[r + 1] = fma2(pack2(__uint_as_float(s[2 * r + 2]), __uint_as_float(s[2 * r + 3])), ks2, m.y);
  }
}

// The same with a factor for each row.
template <bool M>
__device__ __noinline__ void form_scores_by_row(uint32_t taddr, const float* neg_m,
                                                const float* unit, float ks, float ev,
                                                f32x2 (&x)[8]) {
  uint32_t s[16];
  tmem_ld16(taddr, s);
  tmem_ld_wait();
  reg_pin(s);
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    const float m0 = M ? neg_m[2 * r] : ev, m1 = M ? neg_m[2 * r + 1] : ev;
    x[r] = pack2(fmaf(__uint_as_float(s[2 * r]), ks * unit[2 * r], m0),
                 fmaf(__uint_as_float(s[2 * r + 1]), ks * unit[2 * r + 1], m1));
  }
}

// Rows that do not see the key: -inf.
__device__ __forceinline__ void hide_rows(f32x2 (&x)[8], uint32_t hidden) {
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    float2 y = unpack2(x[r]);
    if (hidden >> (2 * r) & 1) y.x = -INFINITY;
    if (hidden >> (2 * r + 1) & 1) y.y = -INFINITY;
    x[r] = pack2(y.x, y.y);
  }
}

// The rare parts of the softmax loop are functions of their own, out of the way
// of its instructions.
// Bit r: row r (mask rows `seen`) does not see draft j.
__device__ __noinline__ uint32_t hidden_rows(const unsigned long long* seen, int j) {
  uint32_t h = 0;
#pragma unroll 4
  for (int r = 0; r < 16; ++r) h |= (seen[r] >> j & 1 ? 0u : 1u) << r;
  return h;
}

// The warp's maximum of each row's s + ev into out[16].
// unit: null where all rows have one factor.
template <bool F8>
__device__ __noinline__ void row_maxima(uint32_t taddr, const float* unit, float ks, float ev,
                                        uint32_t hidden, float* out) {
  const int lane = threadIdx.x & 31;
  f32x2 t[8];
  if (F8 && unit)
    form_scores_by_row<false>(taddr, nullptr, unit, ks, ev, t);
  else
    form_scores<false>(taddr, nullptr, ks, ev, t);
  hide_rows(t, hidden);
  float top = -INFINITY;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float2 y = unpack2(t[r / 2]);
    const float z = redux_max(r & 1 ? y.y : y.x);
    if (lane == r) top = z;
  }
  if (lane < 16) out[lane] = top;
}

// Row r's new reference from the four warps' maxima, and what its sums are
// multiplied by twice: a sum of zero rows' weights may be 2^100 while the reference
// moves by more than the 126 binades of one factor.
template <bool F8, int NR>
__device__ __noinline__ void new_reference(TreeRows<NR>* rows, int r, int have) {
  rows->alpha[r] = 1.0f;
  if (r >= have) return;
  const float top = fmaxf(fmaxf(rows->part[0][r], rows->part[1][r]),
                          fmaxf(rows->part[2][r], rows->part[3][r]));
  const float m_old = rows->m[r];
  const float m_new = fmaxf(m_old, top + (Lazy<F8>::kLog2 - Lazy<F8>::kTop));
  if (m_new == -INFINITY || isnan(rows->neg_m[r])) return;
  rows->m[r] = m_new;
  rows->neg_m[r] = -m_new;
  rows->alpha[r] = ex2_approx(0.5f * (m_old - m_new));
}

// y of four rows of a channel, plus the NaN and infinities of the drafts `bad` that
// the rows see; v: the channel in the value row of draft 0.
template <int D, bool F8>
__device__ __noinline__ float4 add_bad(float4 y, unsigned long long bad,
                                       const unsigned long long* seen, const uint8_t* v) {
#pragma unroll 1
  for (int j = 0; j < 64; ++j) {
    if (!(bad >> j & 1)) continue;
    float z;
    if constexpr (F8)
      z = (v[j * D] & 0x7f) == 0x7f ? NAN : 0.0f;
    else
      z = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(v)[j * D]);
    if (isfinite(z)) continue;
    if (seen[0] >> j & 1) y.x += z;
    if (seen[1] >> j & 1) y.y += z;
    if (seen[2] >> j & 1) y.z += z;
    if (seen[3] >> j & 1) y.w += z;
  }
  return y;
}

// 16 columns of O, `pieces` times `stride` columns apart, times alpha^2.
__device__ __noinline__ void rescale(uint32_t taddr, int pieces, int stride, const float* alpha) {
  tc_fence_after_sync();
#pragma unroll 1
  for (int k = 0; k < pieces; ++k) {
    uint32_t o[16];
    tmem_ld16(taddr + k * stride, o);
    tmem_ld_wait();
    reg_pin(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * (alpha[i] * alpha[i]));
    tmem_st16(taddr + k * stride, o);
  }
  tmem_st_wait();
}

// Barrier `id` of a softmax group with an OR over it.
__device__ __forceinline__ bool group_bar_or(int id, bool any) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(any)), "r"(id), "n"(kTile)
      : "memory");
  return r != 0;
}

template <bool V>
struct Flag {
  static constexpr bool value = V;
};

// PV(i) of the share's tile i is complete (and with it all earlier ones).  Tiles
// alternate between two barriers; a softmax thread at tile `it` knows PV(it - 3) to be
// complete (it wrote P(it - 1) over what that read) and PV(it) not to be, so that the
// parities of PV(it - 1) and PV(it - 2) on their barriers tell them from their neighbours.
__device__ __forceinline__ bool product_done(int i, bool ok, TreeBars* bars, uint32_t code) {
  return ok && t_wait(&bars->pv_done[i & 1], (i >> 1) & 1, bars, code);
}

// ------------------------------------------------------------ the kernel
template <int D, bool F8, int NR>
__global__ void __launch_bounds__(TreeLayout<D, F8, NR>::kThreads, TreeLayout<D, F8, NR>::kCtas)
    fa_tree_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                   const __grid_constant__ TreeParams p) {
  using L = TreeLayout<D, F8, NR>;
  constexpr int kSlots = L::kSlots;
  constexpr int kParts = L::kParts;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  TreeBars* bars = reinterpret_cast<TreeBars*>(smem + L::kBar);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int share = blockIdx.x / p.row_tiles;
  const int rt = blockIdx.x % p.row_tiles;
  // the merge may be launched: it waits for this grid's end before it reads
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (threadIdx.x == 0) {
    mbar_init(&bars->q_ready, L::kSoft);
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&bars->full[s], 1);
      mbar_init(&bars->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars->s_full[s], 1);
      mbar_init(&bars->p_ready[s], L::kSoft / 32);
      mbar_init(&bars->pv_done[s], 1);
    }
    mbar_init(&bars->drain, L::kMmaWarps);
    // an earlier CTA already recorded a pipeline timeout: exit without work
    bars->abort_flag = (*static_cast<volatile unsigned int*>(&g_tree_error) != 0) ? 1 : 0;
    fence_mbar_init();
  }
  // what needs no share comes first, beside the warp that finds it
  if (warp == L::kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == L::kMmaWarp) {
    tmem_alloc(&bars->tmem_base, L::kCols);
    tmem_relinquish();
  }
  if (warp == 0) {
    // the share: units [unit0, unit1) of the list of all pairs
    const int total = all_units(p);
    const int size = share_size(total, p.shares);
    const int unit0 = static_cast<int>(min(static_cast<long long>(share) * size,
                                           static_cast<long long>(total)));
    const int unit1 = min(unit0 + size, total);
    if (lane == 0) {
      bars->unit0 = unit0;
      bars->unit1 = unit1;
      bars->start_u0 = unit1;  // no pair
      bars->start_b = bars->start_h = 0;
    }
    __syncwarp();
    if (unit0 < unit1) {
      int before = 0;  // units of the sequences before this batch of 32
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int nt = b0 + lane < p.B ? seq_tiles(p, b0 + lane) : 0;
        const int n = nt > 0 ? (nt + kPairCost) * p.Hkv : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const int lo = before + incl - n;
        if (n > 0 && unit0 >= lo && unit0 < lo + n) {
          const int h = (unit0 - lo) / (nt + kPairCost);
          const int u0 = lo + h * (nt + kPairCost);
          bars->start_b = b0 + lane;
          bars->start_h = h;
          bars->start_u0 = u0;
          PairInfo& first = bars->pair[0];
          first.b = b0 + lane;
          first.h = h;
          first.bh = static_cast<long long>(b0 + lane) * p.Hkv + h;
          first.u0 = u0;
          first.len = seq_len(p, b0 + lane);
          first.nt = nt;
          first.t0 = max(unit0 - u0 - kPairCost, 0);
          first.tiles = min(nt, unit1 - u0 - kPairCost) - first.t0;
          first.valid = 1;
          first.bad[0] = first.bad[1] = 0;
          first.qmax = -kNoExponent;
          first.qmin = kNoExponent;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
        if (unit0 < before) break;
      }
      __syncwarp();
      const int b = bars->start_b + lane;
      bars->lens[lane] = b < p.B ? seq_len(p, b) : 0;
    }
    if (p.split && rt == 0 && lane == 0) {
      // for the merge: the pair whose second part begins this share
      int4 d = make_int4(-1, 0, 0, 0);
      const PairInfo& first = bars->pair[0];
      if (unit0 < unit1 && first.t0 > 0) {
        const int u = first.u0 + kPairCost;
        if (u / size == share - 1)
          d = make_int4(static_cast<int>(first.bh), share - 1, (u + first.nt - 1) / size, 0);
      }
      p.split[share] = d;
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  if (bars->abort_flag || !Walk(bars).inside()) {
    if (warp == L::kMmaWarp) tmem_dealloc(tmem, L::kCols);
    return;
  }
  // the first pair's queries are asked for before the streams begin
  const int have = min(p.R - rt * kTreeRows, NR);  // query rows of this tile
  const int trow = (rt * kTreeRows + static_cast<int>(threadIdx.x)) % p.T;
  PairLoads<D, NR> in;
  if (warp < L::kTmaWarp) in.load(p, bars->pair[0].b, bars->pair[0].bh, rt, have, trow);
  const uint32_t sRing = smem_u32(smem + L::kRing);

  if (warp == L::kTmaWarp) {
    // ------------------------------------------------ TMA producer
    if (lane == 0) {
      int n = 0;  // slots filled so far
      bool ok = true;
      auto slot = [&]() -> int {
        const int s = n % kSlots;
        if (!(ok = ok && t_wait(&bars->empty[s], ((n / kSlots) & 1) ^ 1, bars, 0x501))) return -1;
        mbar_arrive_expect_tx(&bars->full[s], L::kSlot);
        ++n;
        return s;
      };
      auto load_k = [&](int row0, int bh) {
        if constexpr (F8) {  // the scales of the tile, on their way into L2 meanwhile
          const long long at = static_cast<long long>(bh) * p.cap + row0;
          const int last = min(kTile, p.cap - row0) - 1;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.k_scale + at));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.k_scale + at + last));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.v_scale + at));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.v_scale + at + last));
        }
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
          const int s = slot();
          if (s < 0) return;
#pragma unroll
          for (int x = 0; x < L::kBoxes / kParts; ++x)
            tma_load_3d(smem + L::kRing + s * L::kSlot + x * (kTile * 128), &tk, &bars->full[s],
                        (c + x) * 64, row0, bh);
        }
      };
      auto load_v = [&](int row0, int bh) {
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
          const int s = slot();
          if (s < 0) return;
#pragma unroll
          for (int x = 0; x < L::kBoxes; ++x)  // 64 columns each
            tma_load_3d(smem + L::kRing + s * L::kSlot + x * (L::kVKeys * 128), &tv,
                        &bars->full[s], x * 64, row0 + c * L::kVKeys, bh);
        }
      };
      for (Walk w(bars); ok && w.valid(p, bars); w.next(p)) {
        const int bh = w.b * p.Hkv + w.h, row0 = w.t0 * kTile;
#pragma unroll 1
        for (int t = -2; ok && t < w.n; ++t) {
          if (t >= 0) load_v(row0 + t * kTile, bh);
          if (t + 2 < w.n) load_k(row0 + (t + 2) * kTile, bh);
        }
      }
    }
    __syncwarp();
  } else if (warp >= L::kMmaWarp) {
    // ------------------------------------------------ MMA issuers
    // A whole warp runs the loop on values that are uniform by construction (votes
    // and reductions), so that descriptors live in uniform registers, where the
    // instruction wants them; one elected lane issues.
    const uint32_t sQ = smem_u32(smem + L::kQ);
    const uint32_t sP = smem_u32(smem + L::kP);
    auto issue = [&](auto pv, auto scores) {
      int n = 0, it = 0, seg = 0;  // slots, tiles and pairs done
      bool ok = true;
      for (Walk w(bars); __all_sync(0xffffffffu, ok && w.valid(p, bars)); w.next(p), ++seg) {
        const int tiles = __reduce_max_sync(0xffffffffu, w.n);
        if (!(ok = all_wait(&bars->q_ready, seg & 1, bars, 0x512))) break;
#pragma unroll 1
        for (int t = -2; t < tiles; ++t) {
          const int i = it + t;  // the share's tile
          if (t >= 0 && !(ok = all_wait(&bars->p_ready[i & 1], (i >> 1) & 1, bars, 0x513))) break;
          if (pv.value && t >= 0) {
            // O^T += V^T P^T
            const uint32_t pbase = sP + (i & 1) * L::kPBytes;
            const uint32_t d = tmem + L::kOCol;
            const int first = n + kParts * (2 + t + min(t, tiles - 2));
#pragma unroll 1
            for (int c = 0; c < kParts; ++c) {
              const int s = (first + c) % kSlots;
              if (!(ok = all_wait(&bars->full[s], ((first + c) / kSlots) & 1, bars, 0x514))) break;
              tc_fence_after_sync();
              const uint32_t vbase = sRing + s * L::kSlot;
              if (!elect_one()) continue;
              if constexpr (F8) {
                // all pieces' columns at once; both operands MN-major, P in e5m2
                constexpr uint32_t idesc =
                    idesc_e4m3_f32(D, L::kPPieces * NR) | (3u << 15) | (1u << 10);
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk)
                  umma_ss_f8(d, sdesc<L::kAtom>(vbase + kk * 32 * L::kAtom, 16, 8 * L::kAtom),
                             sdesc<L::kPAtom>(pbase + kk * 32 * L::kPAtom, L::kPBox, 8 * L::kPAtom),
                             idesc,
                             (t > 0 || kk > 0) ? 1u : 0u);
              } else {
                constexpr uint32_t idesc = idesc_bf16_f32(D, NR, true, true);
#pragma unroll
                for (int kk = 0; kk < L::kVKeys / 16; ++kk)
                  umma_ss(d, sdesc_sw128(vbase + kk * 2048, L::kVKeys * 128, 1024),
                          sdesc<L::kPAtom>(pbase + (c * L::kVKeys + kk * 16) * L::kPAtom, 16,
                                           8 * L::kPAtom),
                          idesc, (t > 0 || c > 0 || kk > 0) ? 1u : 0u);
              }
              umma_commit(&bars->empty[s]);
            }
            __syncwarp();
            if (!ok) break;
            if (elect_one()) umma_commit(&bars->pv_done[i & 1]);
          }
          if (scores.value && t + 2 < tiles) {
            // S^T of tile t + 2 = K Q^T, into the buffer that softmax(t) has read
            const uint32_t d = tmem + (i & 1) * NR;
            const int first = n + kParts * (t < 0 ? t + 2 : 2 * t + 3);
#pragma unroll 1
            for (int c = 0; c < kParts; ++c) {
              const int s = (first + c) % kSlots;
              if (!(ok = all_wait(&bars->full[s], ((first + c) / kSlots) & 1, bars, 0x511))) break;
              tc_fence_after_sync();
              const uint32_t kbase = sRing + s * L::kSlot;
              if (!elect_one()) continue;
              if constexpr (F8) {
                constexpr uint32_t idesc = idesc_e4m3_f32(128, NR);
#pragma unroll
                for (int x = 0; x < 2 * (D / 32); ++x) {
                  const int piece = x / (D / 32), kk = x % (D / 32);
                  umma_ss_f8(d, sdesc<L::kAtom>(kbase + kk * 32, 16, 8 * L::kAtom),
                             sdesc<L::kAtom>(sQ + piece * L::kQPiece + kk * 32, 16, 8 * L::kAtom),
                             idesc, x > 0 ? 1u : 0u);
                }
              } else {
                constexpr uint32_t idesc = idesc_bf16_f32(128, NR, false, false);
                constexpr int kSteps = D / 16 / kParts;  // of 16 columns, in this slot
#pragma unroll
                for (int kk = 0; kk < kSteps; ++kk)
                  umma_ss(d, sdesc_sw128(kbase + (kk >> 2) * (kTile * 128) + (kk & 3) * 32, 16, 1024),
                          sdesc_sw128(sQ + (c + (kk >> 2)) * (NR * 128) + (kk & 3) * 32, 16, 1024),
                          idesc, (c > 0 || kk > 0) ? 1u : 0u);
              }
              umma_commit(&bars->empty[s]);
            }
            __syncwarp();
            if (!ok) break;
            if (elect_one()) umma_commit(&bars->s_full[i & 1]);
          }
        }
        n += 2 * kParts * tiles;
        it += tiles;
      }
      __syncwarp();
      if (elect_one()) umma_commit(&bars->drain);
    };
    if constexpr (L::kMmaWarps == 1) {
      issue(Flag<true>{}, Flag<true>{});
    } else if (warp == L::kMmaWarp) {
      issue(Flag<true>{}, Flag<false>{});
    } else {
      issue(Flag<false>{}, Flag<true>{});
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ softmax and epilogue
    // A failed wait clears ok: the warp then skips the work that is left, but
    // none of the barriers, which the four warps pass together.
    const int tid = threadIdx.x;
    const int key = tid % kTile, group = tid / kTile;
    const int quad = warp & 3;  // its tensor-memory lanes: keys, and channels
    const int own = group * 16;  // first of the thread's rows
    const uint32_t tlane = tmem_addr(tmem, quad * 32, 0);
    auto soft_bar = [] { named_bar_sync(1, L::kSoft); };
    TreeRows<NR>* const both = reinterpret_cast<TreeRows<NR>*>(smem + L::kRows);
    int it = 0, seg = 0, n = 0;
    bool ok = true;
    // this thread's scale bytes of the next tile, loaded a tile ahead
    uint32_t kb = 127, vb = 127;
    auto load_scales = [&](long long bh, int pos, int end) {
      kb = vb = 127;
      if (F8 && pos < end) {
        kb = __ldg(p.k_scale + bh * p.cap + pos);
        vb = __ldg(p.v_scale + bh * p.cap + pos);
      }
    };
    f32x2 l[8];             // sums of this key column, by row
    float factor = 0.0f;    // scale log2(e) and the unit of the query pieces, or kByRow
#pragma unroll 1
    for (;; ++seg) {
      // ---- the next pair's queries: S of the last tile is complete, so that Q is
      // free, and the first scores are formed during this pair's epilogue
      PairInfo& next = bars->pair[seg & 3];
      if (next.valid) {
        TreeRows<NR>* const rows = both + (seg & 1);
        if (seg > 0) in.load(p, next.b, next.bh, rt, have, trow);
        load_scales(next.bh, next.t0 * kTile + key, min(next.len + p.T, p.cap));
        if (tid == 0) next_pair(p, bars, next, bars->pair[(seg + 1) & 3]);
        if (seg > 0) ok = product_done(it - 1, ok, bars, 0x526);
        __syncwarp();
        factor = store_queries<D, F8, NR>(smem + L::kQ, rows, in, have, p.scale_log2, &next);
        const unsigned long long any = in.drafts(p);
        if (tid == 0) next.any = any;
        fence_proxy_async_smem();
        mbar_arrive(&bars->q_ready);
      } else if (seg > 0) {
        ok = product_done(it - 1, ok, bars, 0x526);
        __syncwarp();
      }
      if (seg > 0) {
        // ---- epilogue: sums over the keys, then a channel a thread
        TreeRows<NR>* const rows = both + ((seg - 1) & 1);
        const PairInfo& pair = bars->pair[(seg - 1) & 3];
        tc_fence_after_sync();
        {
          float y[16];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 z = unpack2(l[i]);
            y[2 * i] = z.x;
            y[2 * i + 1] = z.y;
          }
          const float z = sum_lanes(y);
          if (lane < 16) rows->part[quad][own + lane] = z;
        }
        soft_bar();
        // partials of a pair that began in an earlier share go to slot 0, of one that
        // goes on in the next to slot 1
        const long long slot =
            pair.tiles == pair.nt ? -1 : 2ll * blockIdx.x + (pair.t0 > 0 ? 0 : 1);
        const long long row0 = pair.bh * p.R + rt * kTreeRows;  // of o and lse
        if (tid < have) {
          const float sum = (rows->part[0][tid] + rows->part[1][tid]) +
                            (rows->part[2][tid] + rows->part[3][tid]);
          const float lse2 = sum == 0.0f ? -INFINITY : __log2f(sum) + rows->m[tid];
          if (ok) {
            if (slot < 0)
              p.lse[row0 + tid] = lse2 * kLn2;
            else
              p.part_lse[slot * p.prow + tid] = lse2;
          }
          rows->inv[tid] = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);
        }
        soft_bar();
        const unsigned long long bad =
            static_cast<unsigned long long>(pair.bad[1]) << 32 | pair.bad[0];
        // channel of this thread: with d = 64 the accumulator's rows are spread over
        // the first 16 lanes of each warp
        const int ch = D == 128 ? key : quad * 16 + lane;
        const bool mine = ok && (D == 128 || lane < 16);
#pragma unroll 1
        for (int r = own; r < min(have, own + 16); r += 4) {
          uint32_t o[4], mid[4], lo[4];
          tmem_ld4(tlane + L::kOCol + r, o);
          if (F8) {
            tmem_ld4(tlane + L::kOCol + NR + r, mid);
            tmem_ld4(tlane + L::kOCol + 2 * NR + r, lo);
          }
          tmem_ld_wait();
          reg_pin(o);
          if (F8) {
            reg_pin(mid);
            reg_pin(lo);
          }
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[i] = __uint_as_float(o[i]);
            if (F8)
              y[i] = fmaf(__uint_as_float(mid[i]) + __uint_as_float(lo[i]), Lazy<F8>::kLowScale, y[i]);
          }
          if (bad) {
            const float4 z = add_bad<D, F8>(
                make_float4(y[0], y[1], y[2], y[3]), bad, rows->seen + r,
                p.v + ((pair.bh * p.cap + pair.len) * D + (mine ? ch : 0)) * (F8 ? 1 : 2));
            y[0] = z.x, y[1] = z.y, y[2] = z.z, y[3] = z.w;
          }
          const float4 inv = *reinterpret_cast<const float4*>(rows->inv + r);
          const float f[4] = {inv.x, inv.y, inv.z, inv.w};
          const long long to = ((slot < 0 ? row0 : slot * p.prow) + r) * D + ch;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (!mine || r + i >= have) continue;
            if (slot < 0)
              p.o[to + i * D] = __float2bfloat16_rn(y[i] * f[i]);
            else
              p.part_o[to + i * D] = y[i] * f[i];
          }
        }
      } else {
        soft_bar();  // the first pair's rows are stored
      }
      if (!next.valid) break;

      // ---- the pair's tiles
      TreeRows<NR>* const rows = both + (seg & 1);
      const long long bh = next.bh;
      const int len = next.len, end = min(len + p.T, p.cap);
      const int tiles = next.tiles;
      int pos = next.t0 * kTile + key;
      {
        const PairInfo& then = bars->pair[(seg + 1) & 3];
        if (then.valid) PairLoads<D, NR>::ask(p, then.b, then.bh, rt, have, trow);
      }
#pragma unroll
      for (int r = 0; r < 8; ++r) l[r] = 0;
      const int first_edge = (len - (pos - key)) / kTile;  // first tile past the committed tokens
#pragma unroll 1
      for (int t = 0; t < tiles; ++t, ++it, pos += kTile) {
        float ks = factor, ev = 0.0f, wv = 1.0f;
        if constexpr (F8) {  // scale log2(e) 2^k_j, e_j as it enters M, and 2^e_j
          // not before here: converted where they are loaded, a tile would wait for them
          asm volatile("" : "+r"(kb), "+r"(vb));
          ks *= __uint_as_float(kb << 23);
          ev = fmaxf(__uint_as_float(0x4b000000u | vb) - 8388735.0f,  // 2^23 + 127
                     Lazy<F8>::kLeastExponent);
          // (a byte of 255, in a draft that was never written, is not an infinity: rows that
          // do not see it have p = 0, and 0 times that is NaN)
          wv = __uint_as_float(min(vb, 254u) << 23);
        }
        if (t + 1 < tiles) load_scales(bh, pos + kTile, end);
        ok = ok && t_wait(&bars->s_full[it & 1], (it >> 1) & 1, bars, 0x522);
        // ---- which rows see this key
        uint32_t hidden = 0;
        if (t >= first_edge) {
          if (pos >= len) hidden = pos < end ? hidden_rows(rows->seen + own, pos - len) : 0xffffu;
          if (hidden == 0xffffu) {  // perhaps never written: finite scales for P = 0
            ks = factor;
            wv = 1.0f;
            ev = 0.0f;
          }
        }
        // ---- x = s - M of this key for the thread's rows
        tc_fence_after_sync();
        const uint32_t scol = tlane + (it & 1) * NR + own;
        float sign = factor;
        asm volatile("" : "+f"(sign));  // one loop for both
        const bool by_row = F8 && sign < 0.0f;
        auto scores = [&](f32x2 (&x)[8]) {
          if (F8 && by_row) {
            f32x2 y[8];
            form_scores_by_row<true>(scol, rows->neg_m + own, rows->unit + own, -ks, 0.0f, y);
#pragma unroll
            for (int r = 0; r < 8; ++r) x[r] = y[r];
          } else {
            form_scores<true>(scol, rows->neg_m + own, ks, 0.0f, x);
          }
        };
        f32x2 x[8];
        scores(x);
        if (hidden) hide_rows(x, hidden);
        float mx = -INFINITY;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float2 y = unpack2(x[r]);
          mx = fmax3f(mx, y.x, y.y);
        }
        if (F8) mx += ev;
        if (group_bar_or(2 + group, mx > Lazy<F8>::kTop)) {
          // ---- some row grew: new references from the maxima over the group's keys
          row_maxima<F8>(scol, by_row ? rows->unit + own : nullptr, by_row ? -ks : ks, ev,
                         hidden, rows->part[quad] + own);
          named_bar_sync(2 + group, kTile);
          if (key < 16) new_reference<F8, NR>(rows, own + key, have);
          named_bar_sync(2 + group, kTile);
          if (t > 0) {
            // PV(it - 1) must be done before O is rescaled
            ok = product_done(it - 1, ok, bars, 0x524);
            __syncwarp();
            rescale(tlane + L::kOCol + own, L::kPPieces, NR, rows->alpha + own);
#pragma unroll
            for (int r = 0; r < 8; r += 2) {
              const ulonglong2 al = *reinterpret_cast<const ulonglong2*>(&rows->alpha[own + 2 * r]);
              l[r] = mul2(mul2(l[r], al.x), al.x);
              l[r + 1] = mul2(mul2(l[r + 1], al.y), al.y);
            }
          }
          scores(x);
          if (hidden) hide_rows(x, hidden);
        }
        // ---- p = 2^x, and P = 2^e p over the P buffer that PV(it - 2) has read.  With one issuing warp
        // it is complete: S(it) was issued behind it.
        if (L::kMmaWarps > 1 && it >= 2) ok = product_done(it - 2, ok, bars, 0x525);
        {
          const f32x2 wv2 = pack2(wv, wv);
          uint32_t hi[8], mid[F8 ? 4 : 1], lo[F8 ? 4 : 1];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 a = unpack2(x[2 * i]), b = unpack2(x[2 * i + 1]);
            const float p0 = ex2_approx(a.x), p1 = ex2_approx(a.y);
            const float p2 = ex2_approx(b.x), p3 = ex2_approx(b.y);
            const f32x2 p01 = pack2(p0, p1), p23 = pack2(p2, p3);
            l[2 * i] = add2(l[2 * i], p01);
            l[2 * i + 1] = add2(l[2 * i + 1], p23);
            if constexpr (F8) {
              const float2 c = unpack2(mul2(p01, wv2)), d = unpack2(mul2(p23, wv2));
              split4(c.x, c.y, d.x, d.y, hi[i], mid[i], lo[i]);
            } else {
              hi[2 * i] = pack_bf16x2(p0, p1);
              hi[2 * i + 1] = pack_bf16x2(p2, p3);
            }
          }
          uint8_t* const at = smem + L::kP + (it & 1) * L::kPBytes;
          if constexpr (F8) {
            *reinterpret_cast<uint4*>(at + L::p_at(key, group)) =
                make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(at + L::p_at(key, L::kGroups + group)) =
                make_uint4(mid[0], mid[1], mid[2], mid[3]);
            *reinterpret_cast<uint4*>(at + L::p_at(key, 2 * L::kGroups + group)) =
                make_uint4(lo[0], lo[1], lo[2], lo[3]);
          } else {
            *reinterpret_cast<uint4*>(at + L::p_at(key, 2 * group)) =
                make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(at + L::p_at(key, 2 * group + 1)) =
                make_uint4(hi[4], hi[5], hi[6], hi[7]);
          }
        }
        if (t >= first_edge) {
          // V(t) in the order of loads.  With S(it) and PV(it - 1) complete, so are
          // all loads that its slot had before: the parity is V(t)'s.
          const int v = n + kParts * (2 + t + min(t, tiles - 2)) + key / L::kVKeys;
          if (t > 0) ok = product_done(it - 1, ok, bars, 0x523);
          ok = ok && t_wait(&bars->full[v % kSlots], (v / kSlots) & 1, bars, 0x521);
          if (ok)
            clean_values<L::kAtom, L::kBoxes, L::kGroups, F8>(
                smem + L::kRing + (v % kSlots) * L::kSlot + (key % L::kVKeys) * L::kAtom,
                L::kVKeys * L::kAtom, key, group, pos, len, end, next.any, next.bad);
        }
        fence_proxy_async_smem();  // P, and cleaned values
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_ready[it & 1]);
      }
      n += 2 * kParts * tiles;
    }
  }

  // ------------------------------------------------ teardown
  if (warp >= L::kMmaWarp) mbar_wait(&bars->drain, 0, &bars->abort_flag, &g_tree_error, 0x5ff);
  if (bars->abort_flag) {
    // let any bulk copy already in flight land before the CTA exits
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000ull) {
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == L::kMmaWarp) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, L::kCols);
  }
}

// ------------------------------------------------------------ merge
// Where several shares cover a pair, its rows' partials are merged.  A block has
// ROWS query rows of a pair and 8 / ROWS warps for each, over the shares.  The pairs
// that are split are at most as many as there are pairs, and as there are ends of shares
// but the last; the grid has the smaller number of them.  Where that is the pairs, a block finds
// its own from the lengths (a few hundred at most) while the shares still run; where
// it is the shares, split[s] names the pair whose second part begins share s.  With a
// block for every pair, each of which added up all lengths, 8 rows x 4 heads of 65536
// sequences of up to 250 tokens took 75 ms; they take 5.2.
constexpr int kMergeThreads = 256;
// The largest weight is 2^-9: a sum of 304 parts of a bf16's largest values stays finite.
constexpr float kMergeRoom = 9.0f;
static_assert(kTreeMaxSms * tree_ctas(1) <= 512, "shares");

__device__ __forceinline__ void load_row(const float* src, float (&x)[4]) {
  const float4 z = *reinterpret_cast<const float4*>(src);
  x[0] = z.x, x[1] = z.y, x[2] = z.z, x[3] = z.w;
}
__device__ __forceinline__ void load_row(const float* src, float (&x)[2]) {
  const float2 z = *reinterpret_cast<const float2*>(src);
  x[0] = z.x, x[1] = z.y;
}

template <int D, int ROWS>
__global__ void __launch_bounds__(kMergeThreads)
    fa_tree_combine(const __grid_constant__ TreeParams p, int blocks) {
  constexpr int kC = D / 32;
  constexpr int kWarps = 8 / ROWS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long bh = blockIdx.x / blocks;
  int first, last;
  if (p.split) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 d = p.split[bh + 1];
    if (d.x < 0) return;
    bh = d.x;
    first = d.y;
    last = d.z;
  } else {
    const int b = static_cast<int>(bh / p.Hkv), h = static_cast<int>(bh % p.Hkv);
    int total = 0, before = 0;
    for (int i = lane; i < p.B; i += 32) {
      const int n = seq_tiles(p, i) + kPairCost;
      total += n;
      if (i < b) before += n;
    }
    const int nt = seq_tiles(p, b);
    total = warp_sum(total) * p.Hkv;
    const int u0 = warp_sum(before) * p.Hkv + (h + 1) * kPairCost + h * nt;  // of its first tile
    const int size = share_size(total, p.shares);
    first = u0 / size;
    last = (u0 + nt - 1) / size;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (first == last) return;
  }
  const int r = static_cast<int>(blockIdx.x % blocks) * ROWS + warp / kWarps;
  const int rt = r / kTreeRows, rs = r % kTreeRows;
  // rows of the partials of share c: slot 1 where the pair begins, else slot 0
  auto slot_row = [&](int c) -> long long {
    return (2ll * (static_cast<long long>(c) * p.row_tiles + rt) + (c == first ? 1 : 0)) * p.prow + rs;
  };
  __shared__ float sm[8], sl[8], so[8][D];
  float m = -INFINITY, l = 0.0f, acc[kC];
#pragma unroll
  for (int k = 0; k < kC; ++k) acc[k] = 0.0f;
  if (r < p.R) {
    // four parts at a time, all of whose loads are under way together
#pragma unroll 1
    for (int c = first + warp % kWarps; c <= last; c += 4 * kWarps) {
      float part[4];
      float x[4][kC];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool there = c + i * kWarps <= last;
        const long long at = slot_row(there ? c + i * kWarps : c);
        part[i] = p.part_lse[at];
        load_row(p.part_o + at * D + lane * kC, x[i]);
        if (!there) part[i] = -INFINITY;
      }
      const float old = m;
      m = fmaxf(m, fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])) + kMergeRoom);
      const float ref = m == -INFINITY ? 0.0f : m;
      const float keep = ex2_approx(old - ref);
      l *= keep;
#pragma unroll
      for (int k = 0; k < kC; ++k) acc[k] *= keep;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (part[i] == -INFINITY) continue;  // no key seen there
        const float w = ex2_approx(part[i] - ref);
        l += w;
#pragma unroll
        for (int k = 0; k < kC; ++k) acc[k] = fmaf(w, x[i][k], acc[k]);
      }
    }
  }
  if constexpr (kWarps > 1) {
#pragma unroll
    for (int k = 0; k < kC; ++k) so[warp][lane * kC + k] = acc[k];
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
    __syncthreads();
    if (warp % kWarps != 0) return;
#pragma unroll
    for (int i = 1; i < kWarps; ++i) m = fmaxf(m, sm[warp + i]);
    const float ref = m == -INFINITY ? 0.0f : m;
    l = 0.0f;
#pragma unroll
    for (int k = 0; k < kC; ++k) acc[k] = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (sl[warp + i] == 0.0f) continue;
      const float w = ex2_approx(sm[warp + i] - ref);
      l = fmaf(w, sl[warp + i], l);
#pragma unroll
      for (int k = 0; k < kC; ++k) acc[k] = fmaf(w, so[warp + i][lane * kC + k], acc[k]);
    }
  }
  if (r < p.R) {
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    const long long row = bh * p.R + r;
#pragma unroll
    for (int k = 0; k < kC; ++k) acc[k] *= inv;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D) + lane * (kC / 2);
    if constexpr (kC == 4)
      *reinterpret_cast<uint2*>(dst) =
          make_uint2(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]));
    else
      *dst = pack_bf16x2(acc[0], acc[1]);
    if (lane == 0) p.lse[row] = l == 0.0f ? -INFINITY : (log2f(l) + (m == -INFINITY ? 0.0f : m)) * kLn2;
  }
}

template <int D, int ROWS>
cudaError_t launch_combine(const TreeParams& p, cudaStream_t s) {
  // launched while the shares still run, for which it waits (griddepcontrol.wait)
  const int blocks = (p.R + ROWS - 1) / ROWS;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(tree_merge_groups(p.B, p.Hkv, p.shares)) * blocks);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fa_tree_combine<D, ROWS>, p, blocks);
}

template <int D, bool F8, int NR>
cudaError_t launch_tile(const TreeParams& p, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t s) {
  constexpr uint32_t smem = TreeLayout<D, F8, NR>::kSmem;
  // once a device (it outlasts the call)
  static std::atomic<unsigned long long> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (!(done.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(fa_tree_kernel<D, F8, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem);
    if (e != cudaSuccess) return e;
    done.fetch_or(bit, std::memory_order_relaxed);
  }
  fa_tree_kernel<D, F8, NR>
      <<<static_cast<unsigned>(p.shares) * p.row_tiles, TreeLayout<D, F8, NR>::kThreads, smem, s>>>(tk, tv, p);
  return cudaGetLastError();
}

template <int D, bool F8>
cudaError_t launch_type(const TreeArgs& a, const CUtensorMap& tk, const CUtensorMap& tv,
                        cudaStream_t s) {
  const TreePlan plan = tree_plan(a.c, a.Hq, a.T, a.num_sms);
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
  p.T = a.T;
  p.R = a.Hq / a.c.Hkv * a.T;
  p.row_tiles = plan.row_tiles;
  p.shares = plan.shares;
  p.prow = plan.prow;
  p.part_o = static_cast<float*>(a.workspace) + 4 * (plan.slots > 0 ? plan.shares : 0);
  p.part_lse = p.part_o + static_cast<size_t>(plan.slots) * plan.prow * D;
  if (plan.slots > 0 && static_cast<long long>(a.c.B) * a.c.Hkv >= plan.shares)
    p.split = static_cast<int4*>(a.workspace);
  p.k_scale = a.c.k_scale;
  p.v_scale = a.c.v_scale;
  p.v = static_cast<const uint8_t*>(a.c.v);
  p.scale_log2 = a.scale * kLog2e;
  const cudaError_t e = p.R <= 16   ? launch_tile<D, F8, 16>(p, tk, tv, s)
                        : p.R <= 32 ? launch_tile<D, F8, 32>(p, tk, tv, s)
                                    : launch_tile<D, F8, 64>(p, tk, tv, s);
  if (e != cudaSuccess || plan.slots == 0) return e;
  // eight rows a block, a warp each, where rows are many or have few parts, else one row.
  // One row and eight, e4m3 calls: 512 rows of 9.5 parts 26.7 and 28.6 us, 1024 of 9.5 26.8
  // and 28.8, 1024 of 4.8 24.8 and 25.4; 2048 of 4.8 51.1 and 48.8, 2048 of 2.4 30.3 and 26.8,
  // 4096 of 2.4 51.5 and 43.5; 1024 of 1.2 parts 26.7 and 26.3.
  const bool few_parts = plan.shares <= 2ll * p.B * p.Hkv;
  return few_parts || static_cast<long long>(p.B) * a.Hq * a.T >= 1536 ? launch_combine<D, 8>(p, s)
                                                                       : launch_combine<D, 1>(p, s);
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
