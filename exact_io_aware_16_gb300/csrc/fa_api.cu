// fa_api.cu — the C ABI of libfa: argument validation, TMA tensor-map
// construction and kernel launches.  No device memory is allocated here.
#include <atomic>
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "../../include/fa.h"
#include "fa_internal.h"
#include "fa_packed.cuh"

namespace {

using EncodeTiledFn = PFN_cuTensorMapEncodeTiled_v12000;

EncodeTiledFn get_encode_tiled() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_shape(int B, int H, int N, int d) { return fa::check_bhnd(B, H, N, d); }

int check_scale(float scale) {
  if (!(scale > 0.0f) || !std::isfinite(scale)) return FA_ERR_SHAPE;
  return FA_OK;
}

// Is the current device an sm_103 part?  Cached per device ordinal.
int check_arch() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return FA_ERR_CUDA;
  static std::atomic<int> cache[64];  // 0 unknown, 1 ok, 2 bad (any thread may fill it)
  if (dev < 64 && cache[dev].load(std::memory_order_relaxed) == 1) return FA_OK;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return FA_ERR_CUDA;
  const bool ok = (major == 10 && minor == 3);
  if (dev < 64) cache[dev].store(ok ? 1 : 2, std::memory_order_relaxed);
  return ok ? FA_OK : FA_ERR_ARCH;
}

// [BH][N][d] bf16 as a 3-D tensor (d, N, BH); box 64 x rows x 1, 128B swizzle.
int encode_bhnd(CUtensorMap* map, const void* base, int BH, int N, int d, int rows) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return FA_ERR_CUDA;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                           static_cast<cuuint64_t>(N) * static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(fa::kBoxCols), static_cast<cuuint32_t>(rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                   strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// A [BH][rows][cols] uint8 (e4m3) tensor as a 3-D tensor (cols, rows, BH);
// box 128 x 128 x 1 (128-byte rows, 128-byte swizzle).  cols must be a
// multiple of 16 (row stride in bytes).
int encode_u8(CUtensorMap* map, const void* base, int BH, int rows, int cols) {
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return FA_ERR_CUDA;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(cols),
                           static_cast<cuuint64_t>(rows) * static_cast<cuuint64_t>(cols)};
  cuuint32_t box[3] = {128, 128, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// A key or value cache as a 3-D tensor (d, cap, B*Hkv) with boxes of `rows`
// tokens, swizzled over the row of the box (128 bytes; 64 for 64 e4m3).
int encode_cache(CUtensorMap* map, const void* base, const fa_cache& c, int rows) {
  const int BH = c.B * c.Hkv;
  if (c.format == FA_CACHE_BF16) return encode_bhnd(map, base, BH, c.cap, c.d, rows);
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return FA_ERR_CUDA;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.cap),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.d),
                           static_cast<cuuint64_t>(c.cap) * static_cast<cuuint64_t>(c.d)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(c.d), static_cast<cuuint32_t>(rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   c.d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// SM count of the current device (cached per device ordinal).
int num_sms() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 1;
  static std::atomic<int> cache[64];
  if (dev < 64) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
    n = 1;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

float log2e_times(float scale) { return static_cast<float>(static_cast<double>(scale) * 1.4426950408889634); }

}  // namespace

extern "C" {

const char* fa_status_string(int status) {
  switch (status) {
    case FA_OK: return "ok";
    case FA_ERR_NULL: return "null pointer";
    case FA_ERR_SHAPE: return "invalid shape, scale or dropout probability";
    case FA_ERR_HEADDIM: return "head dimension must be 64 or 128";
    case FA_ERR_ALIGN: return "pointer not 16-byte aligned";
    case FA_ERR_ARCH: return "device is not sm_103 (GB300)";
    case FA_ERR_WORKSPACE: return "workspace missing or too small";
    case FA_ERR_CUDA: return "CUDA call failed";
    case FA_ERR_DEVICE_TIMEOUT: return "device pipeline wait timed out";
    default: return "unknown status";
  }
}

long long fa_forward_tile_count(int N, int causal) {
  if (N < 1) return 0;
  const long long nq = fa::num_tiles(N, fa::kTileM);
  const long long nk = fa::num_tiles(N, fa::kTileN);
  if (!causal) return nq * nk;
  return nq * (nq + 1) / 2;  // tiles are square: query tile i visits key tiles 0..i
}

static int forward_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int H, int N, int d, float scale, int causal, const uint8_t* bmask,
                        long long mstride, void* stream, const fa::DropArgs* drop = nullptr) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
  int st = check_shape(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  const int BH = B * H;
  fa::TensorMaps maps;
  if (encode_bhnd(&maps.q, q, BH, N, d, 128) != FA_OK ||
      encode_bhnd(&maps.k, k, BH, N, d, 128) != FA_OK ||
      encode_bhnd(&maps.v, v, BH, N, d, 128) != FA_OK)
    return FA_ERR_CUDA;
  fa::FwdArgs a;
  a.tq = &maps.q;
  a.tk = &maps.k;
  a.tv = &maps.v;
  a.o = o;
  a.lse = lse;
  a.BH = BH;
  a.N = N;
  a.d = d;
  a.scale_log2 = log2e_times(scale);
  a.causal = causal ? 1 : 0;
  a.bmask = bmask;
  a.mstride = mstride;
  a.num_sms = num_sms();
  if (drop) {
    a.dropout = true;
    a.drop = *drop;
  }
  cudaError_t e = fa::launch_forward(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// block-sparse calls: mask present, at most kMaxSparseTiles tiles, stride >= 0
static int check_sparse(const uint8_t* bmask, long long mstride, int N) {
  if (!bmask) return FA_ERR_NULL;
  if (N > 128 * fa::kMaxSparseTiles || mstride < 0) return FA_ERR_SHAPE;
  return FA_OK;
}

int fa_forward(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
               int N, int d, float scale, int causal, void* stream) {
  return forward_impl(q, k, v, o, lse, B, H, N, d, scale, causal, nullptr, 0, stream);
}

int fa_forward_blocksparse(const void* q, const void* k, const void* v, void* o, float* lse,
                           int B, int H, int N, int d, float scale, int causal,
                           const uint8_t* block_mask, long long mask_head_stride, void* stream) {
  const int st = check_sparse(block_mask, mask_head_stride, N);
  if (st != FA_OK) return st;
  return forward_impl(q, k, v, o, lse, B, H, N, d, scale, causal, block_mask, mask_head_stride,
                      stream);
}

size_t fa_backward_workspace_size(int B, int H, int N, int d) {
  if (check_shape(B, H, N, d) != FA_OK) return 0;
  const size_t bytes = static_cast<size_t>(B) * H * N * sizeof(float);
  return (bytes + 255) & ~static_cast<size_t>(255);
}

int fa_backward_preprocess(const void* o, const void* dO, float* D, int B, int H, int N, int d,
                           void* stream) {
  if (!o || !dO || !D) return FA_ERR_NULL;
  int st = check_shape(B, H, N, d);
  if (st != FA_OK) return st;
  if (!aligned16(o) || !aligned16(dO) || !aligned16(D)) return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  const long long rows = static_cast<long long>(B) * H * N;
  cudaError_t e = fa::launch_bwd_preprocess(o, dO, D, rows, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

static int bwd_step(const void* q, const void* k, const void* v, const void* dO, const float* lse,
                    float* D, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                    float scale, int causal, void* stream, bool do_dkdv, bool do_dq,
                    const uint8_t* bmask = nullptr, long long mstride = 0,
                    const fa::DropArgs* drop = nullptr) {
  if (!q || !k || !v || !dO || !lse || !D) return FA_ERR_NULL;
  if ((do_dkdv && (!dk || !dv)) || (do_dq && !dq)) return FA_ERR_NULL;
  int st = check_shape(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dO) || !aligned16(lse) ||
      !aligned16(D) || (do_dq && !aligned16(dq)) || (do_dkdv && (!aligned16(dk) || !aligned16(dv))))
    return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  const int BH = B * H;
  fa::TensorMaps maps;
  if (encode_bhnd(&maps.q, q, BH, N, d, 128) != FA_OK ||
      encode_bhnd(&maps.k, k, BH, N, d, 128) != FA_OK ||
      encode_bhnd(&maps.v, v, BH, N, d, 128) != FA_OK ||
      encode_bhnd(&maps.dO, dO, BH, N, d, 128) != FA_OK)
    return FA_ERR_CUDA;
  fa::BwdArgs a;
  a.tq = &maps.q;
  a.tk = &maps.k;
  a.tv = &maps.v;
  a.tdo = &maps.dO;
  a.lse = lse;
  a.D = D;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.BH = BH;
  a.N = N;
  a.d = d;
  a.scale = scale;
  a.scale_log2 = log2e_times(scale);
  a.causal = causal ? 1 : 0;
  a.bmask = bmask;
  a.mstride = mstride;
  a.num_sms = num_sms();
  if (drop) {
    a.dropout = true;
    a.drop = *drop;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // dQ first: it refines D in place (exact D = sum_j P_ij dP_ij), which the
  // dK / dV kernel then reads.
  if (do_dq && fa::launch_bwd_dq(a, s) != cudaSuccess) return FA_ERR_CUDA;
  if (do_dkdv && fa::launch_bwd_dkdv(a, s) != cudaSuccess) return FA_ERR_CUDA;
  return FA_OK;
}

int fa_backward_dkdv(const void* q, const void* k, const void* v, const void* dO,
                     const float* lse, const float* D, void* dk, void* dv, int B, int H, int N,
                     int d, float scale, int causal, void* stream) {
  return bwd_step(q, k, v, dO, lse, const_cast<float*>(D), nullptr, dk, dv, B, H, N, d, scale,
                  causal, stream, true, false);
}

int fa_backward_dq(const void* q, const void* k, const void* v, const void* dO, const float* lse,
                   float* D, void* dq, int B, int H, int N, int d, float scale, int causal,
                   void* stream) {
  return bwd_step(q, k, v, dO, lse, D, dq, nullptr, nullptr, B, H, N, d, scale, causal, stream,
                  false, true);
}

static int backward_impl(const void* q, const void* k, const void* v, const void* o,
                         const void* dO, const float* lse, void* dq, void* dk, void* dv, int B,
                         int H, int N, int d, float scale, int causal, const uint8_t* bmask,
                         long long mstride, void* workspace, size_t workspace_bytes,
                         void* stream, const fa::DropArgs* drop = nullptr) {
  if (!q || !k || !v || !o || !dO || !lse || !dq || !dk || !dv) return FA_ERR_NULL;
  int st = check_shape(B, H, N, d);
  if (st != FA_OK) return st;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!workspace || workspace_bytes < fa_backward_workspace_size(B, H, N, d) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FA_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) ||
      !aligned16(lse) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  float* D = static_cast<float*>(workspace);
  if ((st = fa_backward_preprocess(o, dO, D, B, H, N, d, stream)) != FA_OK) return st;
  return bwd_step(q, k, v, dO, lse, D, dq, dk, dv, B, H, N, d, scale, causal, stream, true, true,
                  bmask, mstride, drop);
}

int fa_backward(const void* q, const void* k, const void* v, const void* o, const void* dO,
                const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                float scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
  return backward_impl(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, nullptr, 0,
                       workspace, workspace_bytes, stream);
}

int fa_backward_blocksparse(const void* q, const void* k, const void* v, const void* o,
                            const void* dO, const float* lse, void* dq, void* dk, void* dv,
                            int B, int H, int N, int d, float scale, int causal,
                            const uint8_t* block_mask, long long mask_head_stride,
                            void* workspace, size_t workspace_bytes, void* stream) {
  const int st = check_sparse(block_mask, mask_head_stride, N);
  if (st != FA_OK) return st;
  return backward_impl(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, block_mask,
                       mask_head_stride, workspace, workspace_bytes, stream);
}

// Dropout parameters of probability p: keep iff the element's 16 random bits
// are >= thr16 = floor(p * 2^16), kept values times the inverse keep
// probability 65536 / (65536 - thr16).  p must lie in [0, 1); thr16 = 0 keeps
// everything and runs the kernels without dropout (*active = false).
static int make_drop(float p, unsigned long long seed, unsigned int offset, fa::DropArgs* out,
                     bool* active) {
  if (!(p >= 0.0f && p < 1.0f)) return FA_ERR_SHAPE;  // also rejects NaN
  const uint32_t thr16 = static_cast<uint32_t>(static_cast<double>(p) * 65536.0);  // floor
  *active = thr16 > 0;
  out->set_seed(static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32));
  out->offset = offset;
  out->thr_hi = thr16 << 16;
  out->rs = static_cast<float>(65536.0 / (65536.0 - thr16));
  return FA_OK;
}

int fa_forward_dropout(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int H, int N, int d, float scale, int causal, float p_drop,
                       unsigned long long seed, unsigned int offset, const uint8_t* block_mask,
                       long long mask_head_stride, void* stream) {
  fa::DropArgs dr;
  bool active = false;
  int st = make_drop(p_drop, seed, offset, &dr, &active);
  if (st != FA_OK) return st;
  if (block_mask && (st = check_sparse(block_mask, mask_head_stride, N)) != FA_OK) return st;
  return forward_impl(q, k, v, o, lse, B, H, N, d, scale, causal, block_mask,
                      block_mask ? mask_head_stride : 0, stream, active ? &dr : nullptr);
}

int fa_backward_dropout(const void* q, const void* k, const void* v, const void* o,
                        const void* dO, const float* lse, void* dq, void* dk, void* dv, int B,
                        int H, int N, int d, float scale, int causal, float p_drop,
                        unsigned long long seed, unsigned int offset, const uint8_t* block_mask,
                        long long mask_head_stride, void* workspace, size_t workspace_bytes,
                        void* stream) {
  fa::DropArgs dr;
  bool active = false;
  int st = make_drop(p_drop, seed, offset, &dr, &active);
  if (st != FA_OK) return st;
  if (block_mask && (st = check_sparse(block_mask, mask_head_stride, N)) != FA_OK) return st;
  return backward_impl(q, k, v, o, dO, lse, dq, dk, dv, B, H, N, d, scale, causal, block_mask,
                       block_mask ? mask_head_stride : 0, workspace, workspace_bytes, stream,
                       active ? &dr : nullptr);
}

int fa_forward_fp8(const void* q8, const void* k8, const void* vt8, float q_descale,
                   float k_descale, float v_descale, void* o, float* lse, int B, int H, int N,
                   int d, float scale, int causal, void* stream) {
  if (!q8 || !k8 || !vt8 || !o || !lse) return FA_ERR_NULL;
  int st = check_shape(B, H, N, d);
  if (st != FA_OK) return st;
  if (d != 128) return FA_ERR_HEADDIM;
  if (N % 16 != 0) return FA_ERR_SHAPE;  // rows of V^T must be 16-byte aligned
  if ((st = check_scale(scale)) != FA_OK || (st = check_scale(q_descale)) != FA_OK ||
      (st = check_scale(k_descale)) != FA_OK || (st = check_scale(v_descale)) != FA_OK)
    return st;
  const double s2 = static_cast<double>(scale) * q_descale * k_descale;
  if (!std::isfinite(s2) || !(s2 > 0.0) || !std::isfinite(static_cast<float>(s2)))
    return FA_ERR_SHAPE;
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(vt8) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  const int BH = B * H;
  fa::TensorMaps maps;
  if (encode_u8(&maps.q, q8, BH, N, d) != FA_OK || encode_u8(&maps.k, k8, BH, N, d) != FA_OK ||
      encode_u8(&maps.v, vt8, BH, d, N) != FA_OK)
    return FA_ERR_CUDA;
  fa::FwdArgs a;
  a.tq = &maps.q;
  a.tk = &maps.k;
  a.tv = &maps.v;
  a.o = o;
  a.lse = lse;
  a.BH = BH;
  a.N = N;
  a.d = d;
  a.scale_log2 = static_cast<float>(s2 * 1.4426950408889634);
  a.causal = causal ? 1 : 0;
  a.fp8 = true;
  a.o_scale = v_descale;
  a.num_sms = num_sms();
  cudaError_t e = fa::launch_forward(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Decode shapes: the cache as for check_bhnd (B*H a TMA coordinate, its key
// tiles an int32 count), and the (head, key range) CTAs of the split kernel
// within an int32 grid.
static int check_decode_shape(int B, int H, int Nq, int Nk, int d) {
  if (Nq < 1 || Nq > fa::kMaxDecodeQueries) return FA_ERR_SHAPE;
  const int st = fa::check_bhnd(B, H, Nk, d);
  if (st != FA_OK) return st;
  const long long BH = static_cast<long long>(B) * H;
  if (BH * fa::decode_splits(BH, Nk) > 0x7fffffffll) return FA_ERR_SHAPE;
  return FA_OK;
}

size_t fa_decode_workspace_size(int B, int H, int Nq, int Nk, int d) {
  if (check_decode_shape(B, H, Nq, Nk, d) != FA_OK) return 0;
  const long long BH = static_cast<long long>(B) * H;
  const long long S = fa::decode_splits(BH, Nk);
  const size_t floats = static_cast<size_t>(BH * S * Nq) * (d + 1);
  return (floats * sizeof(float) + 512 + 255) & ~static_cast<size_t>(255);
}

int fa_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
              int Nq, int Nk, int d, float scale, int causal, void* workspace,
              size_t workspace_bytes, void* stream) {
  if (!q || !k || !v || !o || !lse) return FA_ERR_NULL;
  int st = check_decode_shape(B, H, Nq, Nk, d);
  if (st != FA_OK) return st;
  if (causal && Nk < Nq) return FA_ERR_SHAPE;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!workspace || workspace_bytes < fa_decode_workspace_size(B, H, Nq, Nk, d) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FA_ERR_WORKSPACE;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  fa::DecodeArgs a;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  a.BH = B * H;
  a.Nq = Nq;
  a.Nk = Nk;
  a.d = d;
  a.S = fa::decode_splits_run(a.BH, Nk, num_sms());
  a.chunk = ((Nk + a.S - 1) / a.S + 63) / 64 * 64;
  a.S = (Nk + a.chunk - 1) / a.chunk;  // no empty ranges
  a.scale = scale;
  a.causal = causal ? 1 : 0;
  const size_t n_o = static_cast<size_t>(a.BH) * a.S * Nq * d;
  a.part_o = static_cast<float*>(workspace);
  // partial lse after the partial outputs, 256-byte aligned
  a.part_lse = reinterpret_cast<float*>(
      (reinterpret_cast<uintptr_t>(a.part_o + n_o) + 255) & ~static_cast<uintptr_t>(255));
  fa::TensorMaps maps;
  if (encode_bhnd(&maps.q, q, a.BH, Nq, d, 128) != FA_OK ||
      encode_bhnd(&maps.k64, k, a.BH, Nk, d, 64) != FA_OK ||
      encode_bhnd(&maps.v64, v, a.BH, Nk, d, 64) != FA_OK)
    return FA_ERR_CUDA;
  cudaError_t e =
      fa::launch_decode(a, &maps.q, &maps.k64, &maps.v64, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// The shape and pointer rules of a cache descriptor, in the order of fa.h.
static int check_cache(const fa_cache* c) {
  if (!c || !c->k || !c->v) return FA_ERR_NULL;
  if (c->format != FA_CACHE_BF16 && c->format != FA_CACHE_E4M3) return FA_ERR_SHAPE;
  const bool e4m3 = c->format == FA_CACHE_E4M3;
  if (e4m3 && (!c->k_scale || !c->v_scale)) return FA_ERR_NULL;
  const int st = fa::check_bhnd(c->B, c->Hkv, c->cap, c->d);
  if (st != FA_OK) return st;
  const long long BH = static_cast<long long>(c->B) * c->Hkv;
  if (c->cap > FA_CACHE_MAX_TOKENS || BH * fa::num_tiles(c->cap, 64) > 0x7fffffffll)
    return FA_ERR_SHAPE;
  return FA_OK;
}

static int check_cache_align(const fa_cache* c) {
  if (!aligned16(c->k) || !aligned16(c->v)) return FA_ERR_ALIGN;
  if (c->format == FA_CACHE_E4M3 && (!aligned16(c->k_scale) || !aligned16(c->v_scale)))
    return FA_ERR_ALIGN;
  return FA_OK;
}

static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Rows a sequence of a write or read: at least one, all of them an int32 count.
static int check_cache_rows(const fa_cache* c, int N) {
  if (N < 1) return FA_ERR_SHAPE;
  return static_cast<long long>(c->B) * c->Hkv > (0x3fffffffll / N) ? FA_ERR_SHAPE : FA_OK;
}

int fa_cache_write(const fa_cache* cache, const void* k, const void* v, const int* lens,
                   const int* counts, int N, void* stream) {
  int st = check_cache(cache);
  if (st != FA_OK) return st;
  if (!k || !v || !lens) return FA_ERR_NULL;
  if ((st = check_cache_rows(cache, N)) != FA_OK) return st;
  if ((st = check_cache_align(cache)) != FA_OK) return st;
  if (!aligned16(k) || !aligned16(v) || !aligned4(lens) || !aligned4(counts)) return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  fa::CacheMoveArgs a{};
  a.c = *cache;
  a.in_k = k;
  a.in_v = v;
  a.at = lens;
  a.counts = counts;
  a.N = N;
  return fa::launch_cache_write(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                     : FA_ERR_CUDA;
}

int fa_cache_read(const fa_cache* cache, void* k, void* v, const int* first, const int* counts,
                  int N, void* stream) {
  int st = check_cache(cache);
  if (st != FA_OK) return st;
  if (!k || !v || !counts) return FA_ERR_NULL;
  if ((st = check_cache_rows(cache, N)) != FA_OK) return st;
  if ((st = check_cache_align(cache)) != FA_OK) return st;
  if (!aligned16(k) || !aligned16(v) || !aligned4(first) || !aligned4(counts)) return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  fa::CacheMoveArgs a{};
  a.c = *cache;
  a.out_k = k;
  a.out_v = v;
  a.at = first;
  a.counts = counts;
  a.N = N;
  return fa::launch_cache_read(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                    : FA_ERR_CUDA;
}

int fa_cache_commit(const fa_cache* cache, const int* lens, const int* path,
                    const int* n_accept, int* new_lens, int T, void* stream) {
  int st = check_cache(cache);
  if (st != FA_OK) return st;
  if (!lens || !path || !n_accept || !new_lens) return FA_ERR_NULL;
  if (T < 1 || T > FA_TREE_MAX_DRAFTS) return FA_ERR_SHAPE;
  if ((st = check_cache_align(cache)) != FA_OK) return st;
  if (!aligned4(lens) || !aligned4(path) || !aligned4(n_accept) || !aligned4(new_lens))
    return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  fa::CacheMoveArgs a{};
  a.c = *cache;
  a.at = lens;
  a.counts = n_accept;
  a.path = path;
  a.new_lens = new_lens;
  a.N = T;
  return fa::launch_cache_commit(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

// Query shapes of a tree decode over a valid cache.
static int check_tree_shape(const fa_cache* c, int Hq, int T) {
  if (Hq < 1 || T < 1 || T > FA_TREE_MAX_DRAFTS || Hq % c->Hkv != 0) return FA_ERR_SHAPE;
  if (c->B > fa::kTreeMaxBatch || static_cast<long long>(c->B) * Hq > 0x7fffffffll / T)
    return FA_ERR_SHAPE;
  // the units of the split are an int32 count
  const long long units = fa::num_tiles(c->cap, fa::kTreeTile) + fa::kTreePairCost;
  return static_cast<long long>(c->B) * c->Hkv * units > 0x3fffffffll ? FA_ERR_SHAPE : FA_OK;
}

size_t fa_decode_tree_workspace_size(const fa_cache* cache, int Hq, int T) {
  if (check_cache(cache) != FA_OK || check_tree_shape(cache, Hq, T) != FA_OK) return 0;
  return fa::tree_workspace_bytes(*cache, Hq, T);
}

int fa_decode_tree(const fa_cache* cache, const void* q, const int* lens,
                   const unsigned long long* mask, long long mask_stride, void* o, float* lse,
                   int Hq, int T, float scale, void* workspace, size_t workspace_bytes,
                   void* stream) {
  int st = check_cache(cache);
  if (st != FA_OK) return st;
  if (!q || !lens || !o || !lse) return FA_ERR_NULL;
  if ((st = check_tree_shape(cache, Hq, T)) != FA_OK) return st;
  if (mask && mask_stride != 0 && mask_stride != T) return FA_ERR_SHAPE;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if (!workspace || workspace_bytes < fa::tree_workspace_bytes(*cache, Hq, T) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FA_ERR_WORKSPACE;
  if ((st = check_cache_align(cache)) != FA_OK) return st;
  if (!aligned16(q) || !aligned16(o) || !aligned4(lse) || !aligned4(lens) ||
      (reinterpret_cast<uintptr_t>(mask) & 7u) != 0)
    return FA_ERR_ALIGN;
  if ((st = check_arch()) != FA_OK) return st;
  fa::TreeArgs a{};
  a.c = *cache;
  a.q = q;
  a.lens = lens;
  a.mask = mask;
  a.mask_stride = mask_stride;
  a.o = o;
  a.lse = lse;
  a.workspace = workspace;
  a.Hq = Hq;
  a.T = T;
  a.scale = scale;
  a.num_sms = num_sms();
  CUtensorMap tk, tv;
  const long long rows = static_cast<long long>(Hq) / cache->Hkv * T;
  const int v_keys = fa::tree_v_keys(cache->format == FA_CACHE_BF16, cache->d, rows);
  if (encode_cache(&tk, cache->k, *cache, fa::kTreeTile) != FA_OK ||
      encode_cache(&tv, cache->v, *cache, v_keys) != FA_OK)
    return FA_ERR_CUDA;
  return fa::launch_decode_tree(a, tk, tv, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

// ---------------------------------------------------------------- packed sequences
// A tensor of `heads` heads of B x T token rows as the kernels take it: strides that no
// element depends on put to d.
static int view_heads(const fa_heads* t, int heads, long long B, long long T, int d,
                      fa::HeadsView* v) {
  if (!t || (!t->p && T > 0)) return FA_ERR_NULL;
  if (t->heads != heads || heads < 1) return FA_ERR_SHAPE;
  v->p = t->p;
  v->heads = heads;
  v->head = heads > 1 ? t->head_stride : d;
  v->token = T > 1 ? t->token_stride : d;
  v->batch = B > 1 ? t->batch_stride : 0;
  if (heads > 1 && v->head < d) return FA_ERR_SHAPE;
  if (T > 1 && v->token < d) return FA_ERR_SHAPE;
  // 16 heads of at most 2^35 bytes between rows are a stride that a tensor map takes
  const long long most = 1ll << 34;
  if (v->head > most || v->token > most || v->batch < 0 || v->batch > most) return FA_ERR_SHAPE;
  // no two rows overlap: each axis steps over all that the axes of smaller steps reach
  struct {
    long long step, count;
  } axis[3] = {{v->head, heads}, {v->token, T}, {v->batch, B}};
  std::sort(axis, axis + 3, [](const auto& x, const auto& y) { return x.step < y.step; });
  __int128 reach = d;
  for (const auto& x : axis) {
    if (x.count <= 1) continue;
    if (x.step < reach) return FA_ERR_SHAPE;
    reach += static_cast<__int128>(x.count - 1) * x.step;
  }
  if (!aligned16(t->p) || (v->head & 7) || (v->token & 7) || (v->batch & 7)) return FA_ERR_ALIGN;
  return FA_OK;
}

// Key or value rows as (d, tokens, heads), boxes of 64 columns x TT tokens; query rows
// as (d, P, tokens, head groups of P), boxes of 64 columns x P heads x TT tokens.  128-byte
// swizzle.  A tensor of no tokens gets a map that is never read through.
static int encode_rows(CUtensorMap* map, const fa::HeadsView& t, int tokens, int d, int P, int TT,
                       const void* otherwise) {
  // extents of one token and head (see fa_packed.cuh); the plan sets each sequence's
  EncodeTiledFn enc = get_encode_tiled();
  if (!enc) return FA_ERR_CUDA;
  const cuuint64_t token = static_cast<cuuint64_t>(t.token) * 2, head = static_cast<cuuint64_t>(t.head) * 2;
  const bool q = P > 0;
  cuuint64_t kdims[3] = {static_cast<cuuint64_t>(d), 1, 1};
  cuuint64_t kstrides[2] = {token, head};
  cuuint32_t kbox[3] = {fa::kBoxCols, static_cast<cuuint32_t>(TT), 1};
  cuuint64_t qdims[4] = {static_cast<cuuint64_t>(d), 1, 1, 1};
  cuuint64_t qstrides[3] = {head, token, head * static_cast<cuuint64_t>(P)};
  cuuint32_t qbox[4] = {fa::kBoxCols, static_cast<cuuint32_t>(P), static_cast<cuuint32_t>(TT), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  void* base = const_cast<void*>(tokens > 0 ? t.p : otherwise);
  const CUresult r =
      enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q ? 4 : 3, base, q ? qdims : kdims,
          q ? qstrides : kstrides, q ? qbox : kbox, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_CUDA;
}

// The maps of q, k, v and, for the backward pass, dO.
static int packed_maps(const fa::PackedArgs& a, bool backward, CUtensorMap maps[4]) {
  const fa::PackedTiling t = fa::packed_tiling(a.q.heads, a.k.heads);
  const void* any = a.workspace;
  const int tokens = backward ? t.TT64 : t.TT, keys = backward ? 64 : 128;
  int st = encode_rows(&maps[0], a.q, a.total_q, a.d, t.P, tokens, any);
  if (st == FA_OK) st = encode_rows(&maps[1], a.k, a.total_k, a.d, 0, keys, any);
  if (st == FA_OK) st = encode_rows(&maps[2], a.v, a.total_k, a.d, 0, keys, any);
  if (st == FA_OK && backward) st = encode_rows(&maps[3], a.dO, a.total_q, a.d, t.P, tokens, any);
  return st;
}

static int check_packed(int B, int total_q, int total_k, int Hq, int Hkv, int d) {
  if (B < 1 || B >= (1 << 20) || total_q < 0 || total_k < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
    return FA_ERR_SHAPE;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (Hq * (total_q / 8ll + B) > 0x7fffffffll || Hkv * (total_k / 128ll + B) > 0x7fffffffll)
    return FA_ERR_SHAPE;
  return FA_OK;
}

size_t fa_forward_packed_workspace_size(int B, int total_q, int total_k, int Hq, int Hkv, int d) {
  if (check_packed(B, total_q, total_k, Hq, Hkv, d) != FA_OK) return 0;
  return fa::packed_layout(B, total_q, total_k, Hq, Hkv, false).bytes;
}

size_t fa_backward_packed_workspace_size(int B, int total_q, int total_k, int Hq, int Hkv, int d) {
  if (check_packed(B, total_q, total_k, Hq, Hkv, d) != FA_OK) return 0;
  return fa::packed_layout(B, total_q, total_k, Hq, Hkv, true).bytes;
}

// What both passes check; the views of q, k, v and o.
static int packed_args(const fa_heads* q, const fa_heads* k, const fa_heads* v, const fa_heads* o,
                       const float* lse, const int* cu_q, const int* cu_k, int B, int total_q,
                       int total_k, int d, float scale, int causal, void* workspace,
                       size_t workspace_bytes, bool backward, fa::PackedArgs* a) {
  if (!q || !k || !v || !o || !cu_q || (!lse && total_q > 0)) return FA_ERR_NULL;
  int st = check_packed(B, total_q, total_k, q->heads, k->heads, d);
  if (st != FA_OK) return st;
  if (!cu_k && total_k != total_q) return FA_ERR_SHAPE;
  if ((st = check_scale(scale)) != FA_OK) return st;
  if ((st = view_heads(q, q->heads, 1, total_q, d, &a->q)) != FA_OK ||
      (st = view_heads(k, k->heads, 1, total_k, d, &a->k)) != FA_OK ||
      (st = view_heads(v, k->heads, 1, total_k, d, &a->v)) != FA_OK ||
      (st = view_heads(o, q->heads, 1, total_q, d, &a->o)) != FA_OK)
    return st;
  if (!aligned4(lse) || !aligned4(cu_q) || !aligned4(cu_k)) return FA_ERR_ALIGN;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
      workspace_bytes < fa::packed_layout(B, total_q, total_k, q->heads, k->heads, backward).bytes)
    return FA_ERR_WORKSPACE;
  a->cu_q = cu_q;
  a->cu_k = cu_k ? cu_k : cu_q;
  a->B = B;
  a->total_q = total_q;
  a->total_k = total_k;
  a->d = d;
  a->scale = scale;
  a->causal = causal ? 1 : 0;
  a->workspace = workspace;
  return FA_OK;
}

int fa_forward_packed(const fa_heads* q, const fa_heads* k, const fa_heads* v, const fa_heads* o,
                      float* lse, const int* cu_q, const int* cu_k, int B, int total_q,
                      int total_k, int d, float scale, int causal, void* workspace,
                      size_t workspace_bytes, void* stream) {
  fa::PackedArgs a{};
  int st = packed_args(q, k, v, o, lse, cu_q, cu_k, B, total_q, total_k, d, scale, causal,
                       workspace, workspace_bytes, false, &a);
  if (st != FA_OK) return st;
  if ((st = check_arch()) != FA_OK) return st;
  a.lse = lse;
  a.num_sms = num_sms();
  if (total_q == 0) return FA_OK;
  CUtensorMap maps[4];
  if ((st = packed_maps(a, false, maps)) != FA_OK) return st;
  return fa::launch_forward_packed(a, maps, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int fa_backward_packed(const fa_heads* q, const fa_heads* k, const fa_heads* v, const fa_heads* o,
                       const fa_heads* dO, const float* lse, const fa_heads* dq,
                       const fa_heads* dk, const fa_heads* dv, const int* cu_q, const int* cu_k,
                       int B, int total_q, int total_k, int d, float scale, int causal,
                       void* workspace, size_t workspace_bytes, void* stream) {
  fa::PackedArgs a{};
  if (!dO || !dq || !dk || !dv) return FA_ERR_NULL;
  int st = packed_args(q, k, v, o, lse, cu_q, cu_k, B, total_q, total_k, d, scale, causal,
                       workspace, workspace_bytes, true, &a);
  if (st != FA_OK) return st;
  if ((st = view_heads(dO, q->heads, 1, total_q, d, &a.dO)) != FA_OK ||
      (st = view_heads(dq, q->heads, 1, total_q, d, &a.dq)) != FA_OK ||
      (st = view_heads(dk, k->heads, 1, total_k, d, &a.dk)) != FA_OK ||
      (st = view_heads(dv, k->heads, 1, total_k, d, &a.dv)) != FA_OK)
    return st;
  if ((st = check_arch()) != FA_OK) return st;
  a.lse = const_cast<float*>(lse);
  a.num_sms = num_sms();
  if (total_q == 0 && total_k == 0) return FA_OK;
  CUtensorMap maps[4];
  if ((st = packed_maps(a, true, maps)) != FA_OK) return st;
  return fa::launch_backward_packed(a, maps, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

// ---------------------------------------------------------------- rotation
// The tables hold 64 bits of a turn, more than a double has: numbers as sums of two doubles, after Dekker
// ("A floating-point technique for extending the available precision", 1971), good to about 2^-100 of
// the value.  Every product that is added to something is an explicit fma, so that no compiler
// has one to contract.
struct Twofold {
  double hi, lo;
};
static Twofold tf_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
static Twofold operator+(const Twofold& a, const Twofold& b) {
  const Twofold s = tf_sum(a.hi, b.hi);
  return tf_sum(s.hi, s.lo + (a.lo + b.lo));
}
static Twofold operator*(const Twofold& a, const Twofold& b) {
  const double p = std::fma(a.hi, b.hi, 0.0), e = std::fma(a.hi, b.hi, -p);
  return tf_sum(p, std::fma(a.hi, b.lo, std::fma(a.lo, b.hi, e)));
}
static Twofold operator/(const Twofold& a, const Twofold& b) {
  Twofold q = {a.hi / b.hi, 0.0};
  for (int i = 0; i < 2; ++i) {
    const Twofold r = a + b * Twofold{-q.hi, -q.lo};
    q = q + Twofold{r.hi / b.hi, 0.0};
  }
  return q;
}
static Twofold tf_power(const Twofold& x, int n) {
  Twofold y = {1.0, 0.0};
  for (int i = 0; i < n; ++i) y = y * x;
  return y;
}
// x^(1/n): one step of Newton's method from a root that is right to a double.
static Twofold tf_root(double x, int n) {
  const Twofold r = {std::pow(x, 1.0 / n), 0.0};
  const Twofold q = Twofold{x, 0.0} / tf_power(r, n);
  return r + r * ((q + Twofold{-1.0, 0.0}) / Twofold{static_cast<double>(n), 0.0});
}
static Twofold tf_within_one(const Twofold& x) {
  if (!(x.hi > 0.0)) return {0.0, 0.0};
  return x.hi >= 1.0 ? Twofold{1.0, 0.0} : x;
}

int fa_rotary_table(unsigned long long* turns, int rot, double base, int scaling, double factor,
                    double original, double low, double high) {
  if (!turns) return FA_ERR_NULL;
  if (rot < 16 || rot > 128 || rot % 16 != 0) return FA_ERR_SHAPE;
  if (!(base > 1.0) || !std::isfinite(base)) return FA_ERR_SHAPE;
  if (scaling < FA_SCALE_NONE || scaling > FA_SCALE_INDEX) return FA_ERR_SHAPE;
  const bool blend = scaling == FA_SCALE_TURNS || scaling == FA_SCALE_INDEX;
  if (scaling != FA_SCALE_NONE && (!(factor >= 1.0) || !std::isfinite(factor))) return FA_ERR_SHAPE;
  if (blend && (!(original >= 1.0) || !std::isfinite(original) || !(low > 0.0) || !(high > low) ||
                !std::isfinite(high)))
    return FA_ERR_SHAPE;
  if (scaling == FA_SCALE_BASE && !std::isfinite(base * std::pow(factor, rot / (rot - 2.0)))) return FA_ERR_SHAPE;
  const Twofold one = {1.0, 0.0}, two_pi = {6.283185307179586232, 2.4492935982947063545e-16};
  const int pairs = rot / 2;
  // f_i = step^-i
  Twofold step = tf_root(base, pairs);
  if (scaling == FA_SCALE_BASE) step = step * tf_root(factor, pairs - 1);
  double first = 0.0, last = 1.0;
  if (scaling == FA_SCALE_INDEX) {
    // the pair that makes t turns within the original context: original * base^(-2i/rot) = 2 pi t
    auto pair_of = [&](double t) { return rot * std::log(original / (two_pi.hi * t)) / (2.0 * std::log(base)); };
    first = std::fmax(std::floor(pair_of(high)), 0.0);
    last = std::fmin(std::ceil(pair_of(low)), rot - 1.0);
  }
  Twofold turns_back = two_pi;  // positions a turn, 2 pi / f_i
  for (int i = 0; i < pairs; ++i) {
    Twofold t = one / turns_back;
    turns_back = turns_back * step;
    if (scaling == FA_SCALE_LINEAR) t = t / Twofold{factor, 0.0};
    if (blend) {
      const Twofold g =
          scaling == FA_SCALE_TURNS
              ? (t * Twofold{original, 0.0} + Twofold{-low, 0.0}) / tf_sum(high, -low)
              : one + Twofold{first - i, 0.0} / Twofold{std::fmax(last - first, 1e-3), 0.0};
      const Twofold keep = tf_within_one(g);
      t = t * (keep + (one + Twofold{-keep.hi, -keep.lo}) / Twofold{factor, 0.0});
    }
    // below 2^62 of 2^64; the higher part may be no whole number, the lower one as large as 2^9
    const double hi = std::ldexp(t.hi, 64), whole = std::floor(hi);
    turns[i] = static_cast<unsigned long long>(whole) +
               static_cast<long long>(std::floor((hi - whole) + std::ldexp(t.lo, 64) + 0.5));
  }
  return FA_OK;
}

// What all four calls check; inputs x and, for the norm's backward pass, g.
static int rotary_args(const fa_rotation* r, const fa_heads* const x[2], const fa_heads* const g[2],
                       const fa_heads* const y[2], const int* positions, int B, int N, int d,
                       bool back, fa::RotaryArgs* a) {
  if (!r || !r->turns || !x[0] || !y[0] || (x[1] && !y[1])) return FA_ERR_NULL;
  if (back && (!g[0] || (x[1] && !g[1]))) return FA_ERR_NULL;
  if (d != 64 && d != 128) return FA_ERR_HEADDIM;
  if (r->rot < 16 || r->rot > d || r->rot % 16 != 0 || !std::isfinite(r->amplitude))
    return FA_ERR_SHAPE;
  if (B < 1 || N < 1 || static_cast<long long>(B) * N > 0x7fffffffll) return FA_ERR_SHAPE;
  for (int t = 0; t < 2; ++t) {
    a->x[t].heads = a->g[t].heads = a->y[t].heads = 0;
    if (!x[t]) continue;
    const int heads = x[t]->heads;
    if (heads < 1 || static_cast<long long>(B) * N > 0x7fffffffll / heads) return FA_ERR_SHAPE;
    int st = view_heads(x[t], heads, B, N, d, &a->x[t]);
    if (st == FA_OK) st = view_heads(y[t], heads, B, N, d, &a->y[t]);
    if (st == FA_OK && back) st = view_heads(g[t], heads, B, N, d, &a->g[t]);
    if (st != FA_OK) return st;
  }
  if (!aligned4(positions) || (reinterpret_cast<uintptr_t>(r->turns) & 7u) != 0) return FA_ERR_ALIGN;
  a->positions = positions;
  a->turns = r->turns;
  a->rot = r->rot;
  a->interleaved = r->interleaved != 0;
  a->amplitude = r->amplitude;
  a->tokens = static_cast<long long>(B) * N;
  a->N = N;
  return FA_OK;
}

static int run_rotary(fa::RotaryArgs& a, int mode, int d, void* stream) {
  const int st = check_arch();
  if (st != FA_OK) return st;
  a.num_sms = num_sms();
  return fa::launch_rotary(a, mode, d, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

int fa_rotary(const fa_rotation* r, const fa_heads* q, const fa_heads* k, const fa_heads* q_out,
              const fa_heads* k_out, const int* positions, int B, int N, int d, void* stream) {
  const fa_heads *x[2] = {q, k}, *y[2] = {q_out, k_out};
  fa::RotaryArgs a{};
  const int st = rotary_args(r, x, x, y, positions, B, N, d, false, &a);
  return st != FA_OK ? st : run_rotary(a, 0, d, stream);
}

int fa_rotary_backward(const fa_rotation* r, const fa_heads* dq, const fa_heads* dk,
                       const fa_heads* dq_in, const fa_heads* dk_in, const int* positions, int B,
                       int N, int d, void* stream) {
  const fa_heads *x[2] = {dq, dk}, *y[2] = {dq_in, dk_in};
  fa::RotaryArgs a{};
  const int st = rotary_args(r, x, x, y, positions, B, N, d, false, &a);
  return st != FA_OK ? st : run_rotary(a, 1, d, stream);
}

static int norm_args(const void* q_weight, const void* k_weight, int weight_bf16, float eps,
                     bool keys, fa::RotaryArgs* a) {
  if (!q_weight || (keys && !k_weight)) return FA_ERR_NULL;
  if ((weight_bf16 != 0 && weight_bf16 != 1) || !(eps >= 0.0f) || !std::isfinite(eps))
    return FA_ERR_SHAPE;
  if (!aligned16(q_weight) || (keys && !aligned16(k_weight))) return FA_ERR_ALIGN;
  a->weight[0] = q_weight;
  a->weight[1] = k_weight;
  a->weight_bf16 = weight_bf16 != 0;
  a->eps = eps;
  return FA_OK;
}

int fa_norm_rotary(const fa_rotation* r, const fa_heads* q, const fa_heads* k,
                   const fa_heads* q_out, const fa_heads* k_out, const int* positions,
                   const void* q_weight, const void* k_weight, int weight_bf16, float eps, int B,
                   int N, int d, void* stream) {
  const fa_heads *x[2] = {q, k}, *y[2] = {q_out, k_out};
  fa::RotaryArgs a{};
  int st = rotary_args(r, x, x, y, positions, B, N, d, false, &a);
  if (st == FA_OK) st = norm_args(q_weight, k_weight, weight_bf16, eps, k != nullptr, &a);
  return st != FA_OK ? st : run_rotary(a, 2, d, stream);
}

int fa_norm_rotary_backward(const fa_rotation* r, const fa_heads* dq, const fa_heads* dk,
                            const fa_heads* q, const fa_heads* k, const fa_heads* dq_in,
                            const fa_heads* dk_in, float* dq_weight, float* dk_weight,
                            const int* positions, const void* q_weight, const void* k_weight,
                            int weight_bf16, float eps, int B, int N, int d, void* workspace,
                            size_t workspace_bytes, void* stream) {
  const fa_heads *x[2] = {q, k}, *g[2] = {dq, dk}, *y[2] = {dq_in, dk_in};
  fa::RotaryArgs a{};
  int st = rotary_args(r, x, g, y, positions, B, N, d, true, &a);
  if (st == FA_OK) st = norm_args(q_weight, k_weight, weight_bf16, eps, k != nullptr, &a);
  if (st != FA_OK) return st;
  if (!dq_weight || (k && !dk_weight)) return FA_ERR_NULL;
  if (!aligned16(dq_weight) || (k && !aligned16(dk_weight))) return FA_ERR_ALIGN;
  if (!workspace || workspace_bytes < FA_NORM_WORKSPACE ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FA_ERR_WORKSPACE;
  a.dw[0] = dq_weight;
  a.dw[1] = k ? dk_weight : nullptr;
  a.partial = static_cast<float*>(workspace);
  return run_rotary(a, 3, d, stream);
}

int fa_selftest_wait_timeout(void* stream) {
  const int st = check_arch();
  if (st != FA_OK) return st;
  return fa::launch_selftest_wait(static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                    : FA_ERR_CUDA;
}

int fa_get_device_error(void* stream, uint32_t* detail) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint32_t w_fwd = 0, w_bwd = 0, w_dtc = 0, w_tree = 0, w_packed = 0, w_pbwd = 0, w_st = 0;
  if (fa::fwd_read_clear_error(&w_fwd, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::bwd_read_clear_error(&w_bwd, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::dtc_read_clear_error(&w_dtc, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::tree_read_clear_error(&w_tree, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::packed_read_clear_error(&w_packed, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::packed_bwd_read_clear_error(&w_pbwd, s) != cudaSuccess) return FA_ERR_CUDA;
  if (fa::st_read_clear_error(&w_st, s) != cudaSuccess) return FA_ERR_CUDA;
  // a launch that gave up may have left its work-item counters dirty
  if (w_fwd && fa::fwd_reset_sched(s) != cudaSuccess) return FA_ERR_CUDA;
  if (w_bwd && fa::bwd_reset_sched(s) != cudaSuccess) return FA_ERR_CUDA;
  uint32_t w = 0;
  for (const uint32_t x : {w_fwd, w_bwd, w_dtc, w_tree, w_packed, w_pbwd, w_st})
    if (!w) w = x;
  if (detail) *detail = w;
  return w ? FA_ERR_DEVICE_TIMEOUT : FA_OK;
}

}  // extern "C"
