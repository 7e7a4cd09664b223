// fa_packed.cuh — what the forward and backward kernels over packed sequences share:
// how rows fill tiles, the plan that a first small kernel leaves in the workspace, and how
// the persistent CTAs take their work from it.
//
// Tiles.  A key head serves G query heads, whose rows need the same keys.  A query tile
// of 128 rows therefore holds P heads of 128 / P tokens (P = packed_heads(G), mostly all of the
// group): row r is token r / P, head r % P.  Keys and values are then read once for all
// of them, and a sequence of few tokens fills a tile with its heads.  Rows that P does
// not fill (126 of 128 for P = 7) are zero or not stored.  The backward pass takes query rows
// in boxes of 64 rows, and its 128-row tile is two of them.
//
// Tensor maps.  Every sequence has its own, whose extent ends where the sequence does:
// what lies behind reads as zeros, so that neither NaN nor infinities of a
// neighbour meet a probability of zero in a product.  The plan kernel copies a map
// encoded for one token of one head and puts the sequence's address and extents in
// (tensormap.replace).  Encoded for one token: a map encoded for 128 KB or more makes TMA read for
// rows outside its extents too, near the map's address (512 boxes with 40 of 128 rows inside: 8.7 MB
// from L2, and 4.1 MB this way), which is behind the tensor where a short sequence ends it, and
// need not be mapped.
//
// Work.  The lengths are on the device, so the plan kernel also lists all tiles, longest
// first (a counting sort by key tiles), and persistent CTAs take (tile, head) items off that
// list: longest-job-first over the whole batch, with the heads of a tile, which share
// keys, next to each other.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "fa_internal.h"
#include "sm103_ptx.cuh"

namespace fa {

// One tile of one sequence.
struct PackedEntry {
  int seq, tile;
  int q0, n;  // first query token of the sequence, queries
  int k0, m;  // first key token, keys
  int pad[2];
};
static_assert(sizeof(PackedEntry) == 32, "two 16-byte loads");

struct PackedHeader {
  unsigned next[2];  // items taken of each list
  unsigned count[2];  // entries of each list
};

// How a call's heads and tokens fill tiles.
struct PackedTiling {
  int P;       // query heads a tile
  int TT;      // query tokens a tile of the forward kernel
  int TT64;    // query tokens in 64 rows (backward)
  int heads;   // head groups of P query heads
  int per_kv;  // of them, those of one key head
};

inline PackedTiling packed_tiling(int Hq, int Hkv) {
  PackedTiling t;
  const int G = Hq / Hkv;
  t.P = packed_heads(G);
  t.TT = 128 / t.P;
  t.TT64 = 64 / t.P;
  t.heads = Hq / t.P;
  t.per_kv = G / t.P;
  return t;
}

// Heads taken together.  Where CTAs have many items (16 or more), as many heads as keep what their
// items stream (two tensors, `tokens` rows of d bf16 a head each) in half of the 129 MB L2:
// 65536 tokens, 32 / 8 heads of 128, forward 20.0 -> 19.6 ms, backward 70.9 -> 69.1 ms.  Where
// they have few, all of them, so that the longest tiles of all heads come first: chunks of one
// head cost the dk, dv kernel of 1000 to 8192 tokens, 7 items a CTA, 16 %.
inline int packed_chunk(long long tokens, int d, int heads, long long items, int ctas) {
  if (items < 16ll * ctas) return heads;
  const long long fit = (64ll << 20) / (tokens * d * 4 + 1);
  return static_cast<int>(fit < 1 ? 1 : (fit > heads ? heads : fit));
}

// The workspace: header, four tensor maps a sequence (the forward pass uses three), two
// lists, and the backward pass's D.
struct PackedLayout {
  size_t maps, list[2], D, bytes;
};

inline PackedLayout packed_layout(int B, int total_q, int total_k, int Hq, int Hkv, bool backward) {
  const PackedTiling t = packed_tiling(Hq, Hkv);
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  PackedLayout l;
  l.maps = 256;
  const size_t b = static_cast<size_t>(B);
  l.list[0] = l.maps + up(b * (backward ? 4 : 3) * 128);
  // a forward item is two query tiles, a backward one two boxes of 64 rows
  const size_t q_tiles = static_cast<size_t>(total_q) / (2 * (backward ? t.TT64 : t.TT)) + b;
  l.list[1] = l.list[0] + up(q_tiles * sizeof(PackedEntry));
  const size_t k_tiles = backward ? static_cast<size_t>(total_k) / 128 + b : 0;
  l.D = l.list[1] + up(k_tiles * sizeof(PackedEntry));
  l.bytes = l.D + (backward ? up(static_cast<size_t>(Hq) * total_q * sizeof(float)) : 0);
  return l;
}

struct PackedPlanArgs {
  CUtensorMap map[4];  // q, k, v, dO, with extents of one token and head
  const __nv_bfloat16* base[4];
  long long token[4];  // elements between tokens
  int nmaps;
  int P, groups, Hkv;      // extents: of q and dO (heads of a tile, tiles' heads), of k and v
  const int* cu_q;
  const int* cu_k;
  int B, total_q, total_k;
  int causal;
  int q_span, k_span;  // query tokens an entry of list 0, key tokens one of list 1
  int TT64;     // query tokens in 64 rows (costs of list 1)
  int nlists;
  unsigned most[2];  // entries the lists have room for
  int shift[2];      // cost to bucket
  PackedHeader* header;
  CUtensorMap* maps;
  PackedEntry* list[2];
};

// Launches `kern` (one CTA an SM, all of its shared memory dynamic) while the kernel before it in the stream
// still runs, for which it waits itself (griddepcontrol.wait).  `ready` says for which
// devices the shared memory has been asked for: that call is as long as a launch.
template <typename Kern, typename Params>
cudaError_t launch_behind(Kern kern, const Params& p, unsigned blocks, unsigned threads, uint32_t smem,
                          std::atomic<unsigned long long>& ready, cudaStream_t s) {
  if (blocks == 0) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(blocks);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, p);
}

cudaError_t launch_packed_plan(const PackedArgs& a, const CUtensorMap* maps, int nmaps, bool backward,
                               cudaStream_t s);

// ---------------------------------------------------------------- device side
// Keys that query token `tok` of a sequence sees.
__device__ __forceinline__ int packed_keys(int tok, int n, int m, bool causal) {
  return causal ? min(max(tok + 1 + m - n, 0), m) : m;
}

// Waits for the launch before this one (the plan), whose writes are then visible.
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The tensor map at `map` was written by generic stores of an earlier kernel.
__device__ __forceinline__ void tensormap_acquire(const CUtensorMap* map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(
                   reinterpret_cast<uint64_t>(map))
               : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// One lane of a converged warp (the same one each time).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// The value of the first lane, which the compiler knows to be the same in all.
__device__ __forceinline__ int uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// An item as the roles of a CTA see it: a list entry and one of its heads.
struct alignas(16) PackedItem {
  PackedEntry e;
  int head;  // of PackedTiling::heads, or (dK/dV) key head; -1: no more items
  int pad[3];
};
static_assert(sizeof(PackedItem) == 48, "three 16-byte stores");

constexpr int kPackedRing = 4;  // items in flight between the roles of a CTA

// The next item of a list (one thread): chunks of `chunk` of the `heads` heads one after the
// other, in each all tiles in the list's order, the chunk's heads of a tile next to each other.
__device__ __forceinline__ PackedItem packed_claim(PackedHeader* h, const PackedEntry* list, int which,
                                                   int heads, int chunk) {
  PackedItem it;
  const unsigned c = atomicAdd(&h->next[which], 1u), count = h->count[which];
  it.head = -1;
  if (c >= count * static_cast<unsigned>(heads)) return it;
  const unsigned before = c / (count * chunk) * chunk;  // heads of earlier chunks
  const unsigned here = min(static_cast<unsigned>(chunk), heads - before);
  const unsigned r = c - before * count, entry = r / here;
  it.head = static_cast<int>(before + r - entry * here);
  const int4* p = reinterpret_cast<const int4*>(list + entry);
  const int4 x = p[0], y = p[1];
  it.e = {x.x, x.y, x.z, x.w, y.x, y.y, {0, 0}};
  return it;
}

}  // namespace fa
