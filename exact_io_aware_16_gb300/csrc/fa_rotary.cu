// fa_rotary.cu — rotation of queries and keys by their positions, with or without a
// norm of each head before it, forward and backward.
//
// Rows of d bf16 (a token's head) pass through once: 2 d bytes in, 2 d bytes out and a
// few operations an element, so every call is bound by memory, and the small ones by
// the launch.  d / 16 lanes hold a row, sixteen elements each as two 16-byte
// chunks chosen so that both members of a pair lie in one lane: the chunks at 8 s
// and rot / 2 + 8 s of lane s where pairs are (i, i + rot / 2), otherwise the two
// halves of elements 16 s .. 16 s + 15.  Either way lane s needs the angles of
// pairs 8 s .. 8 s + 7 and nothing from its neighbours.
//
// Measured, 16384 tokens of 32 and 8 heads of 128 (335 MB in and out): the rotation 53 us,
// 6.3 TB/s, as fast as a copy; with the norm 60 us, 5.6 TB/s, where the lanes' arithmetic and
// shuffles fill two thirds of the issue slots; the norm's backward pass (503 MB) 93 us and 5 us for
// the weights' gradients, 5.4 TB/s. The next tokens of some sequences take 4 us.
//
// Angles: position * turns[i] modulo 2^64 is the exact angle in units of 2^-64 turns
// (the table holds f_i / 2 pi to 2^-65), and its upper 32 bits, read as signed, are the
// angle in (-1/2, 1/2] turns.  sincospif of twice that needs no range reduction; all
// of it is off by about 2^-23, however far the position.
#include <algorithm>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kWarps = kRotaryThreads / 32;

struct Row16 {
  uint4 a, b;  // the lane's two chunks of eight bf16
};

__device__ __forceinline__ void unpack8(const uint4& x, float (&f)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a lane's chunks lie in a row, and whether they turn.
struct LaneMap {
  int a, b;
  bool turns, half;
};

template <int D>
__device__ __forceinline__ LaneMap lane_map(int sub, const RotaryArgs& p) {
  LaneMap m;
  m.turns = sub < p.rot / 16;
  m.half = m.turns && !p.interleaved;
  m.a = m.half ? 8 * sub : 16 * sub;
  m.b = m.half ? p.rot / 2 + 8 * sub : 16 * sub + 8;
  return m;
}

// Cosines and sines (times the amplitude) of pairs 8 sub .. 8 sub + 7 at position
// `pos`.  The 32 * 16 / D row groups of the warp find an equal share each and hand
// the others theirs.
template <int D>
__device__ __forceinline__ void lane_angles(const RotaryArgs& p, const LaneMap& m, int sub, int grp,
                                            int pos, float (&c)[8], float (&s)[8]) {
  constexpr int L = D / 16, E = 8 * L / 32;  // lanes a row, pairs a lane
  float mc[E], ms[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    mc[e] = 1.0f;
    ms[e] = 0.0f;
    if (m.turns) {
      const unsigned long long turn = p.turns[8 * sub + E * grp + e];
      const unsigned long long at = static_cast<unsigned long long>(static_cast<long long>(pos)) * turn;
      const float x = static_cast<float>(static_cast<int>(at >> 32)) * 0x1p-31f;  // half turns
      sincospif(x, &ms[e], &mc[e]);
      mc[e] *= p.amplitude;
      ms[e] *= p.amplitude;
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = __shfl_sync(0xffffffffu, mc[j % E], (j / E) * L + sub);
    s[j] = __shfl_sync(0xffffffffu, ms[j % E], (j / E) * L + sub);
  }
}

// Turns the lane's eight pairs; `sign` -1: backwards.
__device__ __forceinline__ void turn(const LaneMap& m, float (&a)[8], float (&b)[8],
                                     const float (&c)[8], const float (&s)[8], float sign) {
  if (!m.turns) return;
  if (m.half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = a[j], y = b[j], sj = sign * s[j];
      a[j] = x * c[j] - y * sj;
      b[j] = y * c[j] + x * sj;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float x = a[2 * j], y = a[2 * j + 1], sj = sign * s[j];
      a[2 * j] = x * c[j] - y * sj;
      a[2 * j + 1] = y * c[j] + x * sj;
      x = b[2 * j];
      y = b[2 * j + 1];
      sj = sign * s[4 + j];
      b[2 * j] = x * c[4 + j] - y * sj;
      b[2 * j + 1] = y * c[4 + j] + x * sj;
    }
  }
}

template <int L>
__device__ __forceinline__ float row_sum(float x, unsigned lanes = 0xffffffffu) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) x += __shfl_xor_sync(lanes, x, o);
  return x;
}

// A row's mean square leaves fp32 above 2^120 (and below 2^-100, where eps does not hide it): the
// power of two that brings the larger of its greatest element and sqrt(eps) to about one.
template <int L>
__device__ __noinline__ float row_scale(float most, float eps, unsigned lanes) {
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(lanes, most, o));
  most = fmaxf(most, sqrtf(eps));
  if (!(most > 0.0f && most < INFINITY)) return 1.0f;
  const int e = (__float_as_int(most) >> 23) - 127;
  return __int_as_float((127 - min(max(e, -126), 126)) << 23);
}

__device__ __forceinline__ void load_weight8(const RotaryArgs& p, int t, int at, float (&w)[8]) {
  if (p.weight_bf16) {
    unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.weight[t]) + at), w);
  } else {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p.weight[t]) + at);
    const float4 x = q[0], y = q[1];
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  }
}

constexpr int blocks_per_sm(int mode) { return mode == 3 ? 2 : (mode == 2 ? 3 : 4); }

// A unit of work is a token's heads of one tensor, or (few tokens) an equal part of them; the
// units of q come before those of k, and warps take them in turn, so that a warp changes the
// tensor once and holds one set of weights, and of sums of their gradients, at a time.  A step is
// 32 * 16 / d heads; the rows of the next are asked for before those of one are worked on.
// MODE 0: rotation, 1: rotation backwards, 2: norm and rotation, 3: its backward pass.
template <int D, int MODE>
__global__ void __launch_bounds__(kRotaryThreads, blocks_per_sm(MODE))
    fa_rotary_kernel(const __grid_constant__ RotaryArgs p) {
  constexpr int L = D / 16, R = 32 / L;  // lanes a row, rows a step
  constexpr bool kNorm = MODE >= 2, kBack = MODE == 3;
  constexpr float kSign = (MODE & 1) ? -1.0f : 1.0f;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % L, grp = lane / L;
  const LaneMap m = lane_map<D>(sub, p);
  if (kBack) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float part_s[kBack ? kWarps : 1][2][D];
  const long long stride = static_cast<long long>(gridDim.x) * kWarps;
  long long u = static_cast<long long>(blockIdx.x) * kWarps + warp, done = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const HeadsView& tx = p.x[t];
    const HeadsView& tg = p.g[t];
    const HeadsView& ty = p.y[t];
    const long long units = p.tokens * p.parts[t];
    float wa[8], wb[8], da[8], db[8];  // weights, and sums of their gradients
    if (kNorm && u - done < units) {
      load_weight8(p, t, m.a, wa);
      load_weight8(p, t, m.b, wb);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) da[j] = db[j] = 0.0f;
    for (; u - done < units; u += stride) {
      const long long v = u - done, tok = v / p.parts[t];
      const int part = static_cast<int>(v - tok * p.parts[t]);
      const long long b = tok / p.N, i = tok - b * p.N;
      const __nv_bfloat16* xr = static_cast<const __nv_bfloat16*>(tx.p) + b * tx.batch + i * tx.token;
      const __nv_bfloat16* gr = static_cast<const __nv_bfloat16*>(tg.p) + b * tg.batch + i * tg.token;
      __nv_bfloat16* yr = static_cast<__nv_bfloat16*>(const_cast<void*>(ty.p)) + b * ty.batch + i * ty.token;
      Row16 x, g;  // of the next step
      auto ask = [&](int h) {
        x.a = x.b = g.a = g.b = make_uint4(0, 0, 0, 0);
        if (h < tx.heads) {
          x.a = *reinterpret_cast<const uint4*>(xr + h * tx.head + m.a);
          x.b = *reinterpret_cast<const uint4*>(xr + h * tx.head + m.b);
          if (kBack) {
            g.a = *reinterpret_cast<const uint4*>(gr + h * tg.head + m.a);
            g.b = *reinterpret_cast<const uint4*>(gr + h * tg.head + m.b);
          }
        }
      };
      const int step = p.parts[t] * R;
      ask(part * R + grp);
      const int pos = p.positions ? p.positions[tok] : static_cast<int>(i);
      float c[8], s[8];
      lane_angles<D>(p, m, sub, grp, pos, c, s);
      for (int h0 = part * R; h0 < tx.heads; h0 += step) {
        const int h = h0 + grp;
        const bool on = h < tx.heads;
        float xa[8], xb[8], ga[8], gb[8];
        unpack8(x.a, xa);
        unpack8(x.b, xb);
        if (kBack) {
          unpack8(g.a, ga);
          unpack8(g.b, gb);
        }
        if (h0 + step < tx.heads) ask(h + step);
        if (kNorm) {
          float ss = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss = fmaf(xa[j], xa[j], fmaf(xb[j], xb[j], ss));
          ss = row_sum<L>(ss);
          float scale = 1.0f;
          if (!(ss <= 0x1p120f && (ss >= 0x1p-100f || p.eps >= 0x1p-76f))) {  // (all lanes of a row)
            float most = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) most = fmaxf(most, fmaxf(fabsf(xa[j]), fabsf(xb[j])));
            const unsigned lanes = ((1u << L) - 1u) << (lane & ~(L - 1));
            scale = row_scale<L>(most, p.eps, lanes);
            ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              xa[j] *= scale;
              xb[j] *= scale;
              ss = fmaf(xa[j], xa[j], fmaf(xb[j], xb[j], ss));
            }
            ss = row_sum<L>(ss, lanes);
          }
          float r = 1.0f / sqrtf(ss * (1.0f / D) + p.eps * scale * scale);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            xa[j] *= r;
            xb[j] *= r;
          }
          if (kBack) {
            r *= scale;
            turn(m, ga, gb, c, s, kSign);
            float dot = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (on) {
                da[j] = fmaf(ga[j], xa[j], da[j]);
                db[j] = fmaf(gb[j], xb[j], db[j]);
              }
              ga[j] *= wa[j];
              gb[j] *= wb[j];
              dot = fmaf(ga[j], xa[j], fmaf(gb[j], xb[j], dot));
            }
            const float mean = row_sum<L>(dot) * (1.0f / D);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              xa[j] = r * (ga[j] - xa[j] * mean);
              xb[j] = r * (gb[j] - xb[j] * mean);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              xa[j] *= wa[j];
              xb[j] *= wb[j];
            }
          }
        }
        if (!kBack) turn(m, xa, xb, c, s, kSign);
        if (on) {
          *reinterpret_cast<uint4*>(yr + h * ty.head + m.a) = pack8(xa);
          *reinterpret_cast<uint4*>(yr + h * ty.head + m.b) = pack8(xb);
        }
      }
    }
    done += units;
    if (kBack) {  // over the row groups of the warp
#pragma unroll
      for (int j = 0; j < 8; ++j) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1) {
          da[j] += __shfl_xor_sync(0xffffffffu, da[j], o);
          db[j] += __shfl_xor_sync(0xffffffffu, db[j], o);
        }
        if (grp == 0) {
          part_s[kBack ? warp : 0][t][m.a + j] = da[j];
          part_s[kBack ? warp : 0][t][m.b + j] = db[j];
        }
      }
    }
  }
  if (kBack) {  // over the block's warps in order
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += kRotaryThreads) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += part_s[kBack ? w : 0][e / D][e % D];
      p.partial[static_cast<size_t>(blockIdx.x) * 2 * D + e] = v;
    }
  }
}

// dw[t][c] = sum over blocks of partial[block][t][c], in a fixed order.
template <int D>
__global__ void __launch_bounds__(256) fa_norm_weight_kernel(const float* __restrict__ partial,
                                                             int blocks, float* dwq, float* dwk) {
  // eight columns a block, 32 slices of the blocks each
  const int col = blockIdx.x * 8 + (threadIdx.x & 7), slice = threadIdx.x >> 3;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float v = 0.0f;
  for (int b = slice; b < blocks; b += 32) v += partial[static_cast<size_t>(b) * 2 * D + col];
  __shared__ float s[32][8];
  s[slice][threadIdx.x & 7] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) sum += s[k][threadIdx.x];
    float* out = col < D ? dwq : dwk;
    if (out) out[col < D ? col : col - D] = sum;
  }
}

template <int D, int MODE>
cudaError_t launch_t(RotaryArgs a, cudaStream_t s) {
  // parts a token's heads are split into: one where the tokens alone fill the GPU's warps, as many
  // as there are steps otherwise
  constexpr int R = 32 * 16 / D;
  long long units = 0;
  for (int t = 0; t < 2; ++t) {
    const long long most = (a.x[t].heads + R - 1) / R, want = (a.num_sms * 32ll + a.tokens - 1) / a.tokens;
    a.parts[t] = static_cast<int>(want < most ? want : most);
    units += a.tokens * a.parts[t];
  }
  const long long blocks = (units + kWarps - 1) / kWarps;
  // as many blocks as run at once (of the backward pass each leaves a partial sum)
  const long long most = static_cast<long long>(a.num_sms) * blocks_per_sm(MODE);
  const unsigned grid =
      static_cast<unsigned>(std::min(blocks, MODE == 3 ? std::min<long long>(most, kNormMaxBlocks) : most));
  fa_rotary_kernel<D, MODE><<<grid, kRotaryThreads, 0, s>>>(a);
  if (MODE == 3) {
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // launched while the blocks still run, for which it waits (griddepcontrol.wait)
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * D / 8);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa_norm_weight_kernel<D>, static_cast<const float*>(a.partial),
                              static_cast<int>(grid), a.dw[0], a.dw[1]);
  }
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_d(const RotaryArgs& a, int mode, cudaStream_t s) {
  switch (mode) {
    case 0: return launch_t<D, 0>(a, s);
    case 1: return launch_t<D, 1>(a, s);
    case 2: return launch_t<D, 2>(a, s);
    default: return launch_t<D, 3>(a, s);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int mode, int d, cudaStream_t s) {
  return d == 64 ? launch_d<64>(a, mode, s) : launch_d<128>(a, mode, s);
}

}  // namespace fa
