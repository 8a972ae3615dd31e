// swin_heads.cuh -- the kernel of swin_heads.cu: norm of every head and rotary
// positions, forward and backward. Included by one translation unit per type.
#pragma once
#include <algorithm>
#include <cstdint>

#include "../../include/swin_attn.h"
#include "swin_calls.cuh"
#include "swin_vec8.cuh"

namespace swin {
namespace heads {

using namespace rows;

constexpr int kMaxPairs = 128;

// n / d for 0 <= n < 2^31: with l = ceil(log2 d) and m = floor(2^(31 + l) / d) + 1 the
// product n m / 2^(31 + l) exceeds n / d by less than 1 / d (Granlund and Montgomery,
// "Division by invariant integers using multiplication", 1994).
struct FastDiv {
  uint32_t d, m, shift;
  static FastDiv by(uint32_t d) {
    uint32_t l = 0;
    while ((uint64_t(1) << l) < d) ++l;
    return {d, (uint32_t)((uint64_t(1) << (31 + l)) / d + 1), 31 + l};
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> shift); }
};

struct Part {
  const uint8_t *x, *dy;  // a part that only turns its gradient has that in x
  uint8_t *out;
  int64_t x_stride, dy_stride, out_stride;  // bytes
  int heads, kind, rot;                     // kind: SWIN_NORM_*; rot: values that turn
  int tile_rows, chunks;                    // rows of a tile; chunks of kItems heads where a row has more
  FastDiv by_heads;                         // heads of a chunk
  float eps;
  const float *gamma, *beta;
  float *sums, *dgamma, *dbeta;  // sums: [ctas][2][hd], or NULL
  int cta0, ctas;                // a multiple of chunks
  bool wide_x, wide_dy, wide_out;  // fp32: 32-byte pieces
};

struct Args {
  int rows, hd, ndim, count, layout;
  int table;  // floats of one of a tile's two tables
  int pair_lanes;  // threads that share a token's pairs in filling it (a power of two)
  FastDiv by_tokens, stride[3], extent[3];
  float amplitude;
  const void *positions;
  int position_bits, shared;
  Part parts[SWIN_HEAD_PARTS_MAX];
  uint64_t freq[kMaxPairs];
  uint8_t axis[kMaxPairs];
};

// Threads of a CTA, items (a head of a token) that each takes at a time, CTAs an SM. The
// next tile's loads wait in registers, 32 bytes a bf16 item and tensor, 64 an fp32 one, so
// registers and bytes in flight pull at one another: forward 512 threads an SM with 64
// bytes each (768 spilled: 1 179 648 x 24 heads of 32 bf16, normed, 1074 us, so 607),
// backward 384 with 128 (1 179 648 x 24 heads, normed, 776 us; 512 with 64 856; fp32
// 65 522 x 36 heads, LayerNorm with beta, 136; 512 with 128 spilled, 202).
constexpr int threads_of(bool bwd) { return bwd ? 192 : 256; }
constexpr int items_of(int bytes) { return bytes == 4 ? 1 : 2; }
constexpr int kBlocks = 2;
constexpr int kParamFloats = 256;  // gamma, as the lanes read it

// ---- the table of a tile -------------------------------------------------------------
// [token][4][rot / 16] quads of floats: a lane v that turns values reads four quads,
// the cosines of its first and of its second vector's pairs, then the sines. The
// rows are 5 rot / 16 quads apart, so that lanes of several tokens meet few banks.
__host__ __device__ constexpr int table_row(int rot16) { return 20 * rot16; }  // floats

// The pair that a thread fills in: its place in a token's row, its frequency and axis.
struct Filler {
  int token, tokens, at, axis;  // first token, tokens a pass (0: nothing to do)
  uint64_t freq;
  template <int kThreads>
  __device__ __forceinline__ void init(const Args &a, int rot) {
    const int rot16 = rot >> 4, pair = threadIdx.x & (a.pair_lanes - 1);
    token = threadIdx.x / a.pair_lanes;
    tokens = kThreads / a.pair_lanes;
    if (pair >= rot >> 1 || token >= tokens) token = 1 << 30;
    const int p = min(pair, kMaxPairs - 1);
    axis = a.axis[p];
    freq = a.freq[p];
    int v, j;
    if (a.layout == SWIN_ROTARY_HALF) {
      v = pair >> 3;
      j = (pair >> 2) & 1;
    } else {
      j = (pair >> 2) >= rot16;
      v = (pair >> 2) - j * rot16;
    }
    at = (j * rot16 + v) * 4 + (pair & 3);
  }
  // Cosines and sines of `count` rows from row t0 on, times the amplitude.
  __device__ __forceinline__ void fill(const Args &a, int rot16, uint32_t t0, int count, float *table) const {
    for (int t = token; t < count; t += tokens) {
      const uint32_t row = t0 + t;
      if (row >= (uint32_t)a.rows) break;
      const uint32_t tok = row - a.by_tokens.div(row) * a.by_tokens.d;
      uint64_t turn;
      if (a.position_bits == 0) {
        uint32_t c = a.stride[axis].div(tok);
        c -= a.extent[axis].div(c) * a.extent[axis].d;
        turn = c * freq;
      } else {
        const int64_t i = (int64_t)(a.shared ? tok : row) * a.ndim + axis;
        turn = (uint64_t)(a.position_bits == 64 ? static_cast<const int64_t *>(a.positions)[i]
                                                : (int64_t) static_cast<const int32_t *>(a.positions)[i]) * freq;
      }
      // the fraction of a turn, of which 32 bits are kept: half turns from -1 to 1
      const float half_turns = (float)(int32_t)(uint32_t)(turn >> 32) * 0x1p-31f;
      float s, c;
      sincospif(half_turns, &s, &c);
      float *to = table + t * table_row(rot16) + at;
      to[0] = c * a.amplitude;
      to[8 * rot16] = s * a.amplitude;
    }
  }
};

// Turns a lane's two vectors by its quads (of the 16 values' 8 pairs).
__device__ __forceinline__ void turn(float2 (&f)[8], int layout, const float *quads, int rot16) {
  float2 c[4], s[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float4 x = *reinterpret_cast<const float4 *>(quads + j * rot16 * 4);
    const float4 y = *reinterpret_cast<const float4 *>(quads + (j + 2) * rot16 * 4);
    c[2 * j] = make_float2(x.x, x.y), c[2 * j + 1] = make_float2(x.z, x.w);
    s[2 * j] = make_float2(y.x, y.y), s[2 * j + 1] = make_float2(y.z, y.w);
  }
  if (layout == SWIN_ROTARY_HALF) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = f[e], b = f[e + 4];
      f[e] = fma(a, c[e], mul(b, make_float2(-s[e].x, -s[e].y)));
      f[e + 4] = fma(a, s[e], mul(b, c[e]));
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float ce = e & 1 ? c[e >> 1].y : c[e >> 1].x, se = e & 1 ? s[e >> 1].y : s[e >> 1].x;
      f[e] = make_float2(fmaf(f[e].x, ce, -f[e].y * se), fmaf(f[e].x, se, f[e].y * ce));
    }
  }
}

// Over the LPH lanes of a head.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float total(const float2 (&u)[8]) {
  float2 s = add(u[0], u[1]);
#pragma unroll
  for (int e = 2; e < 8; ++e) s = add(s, u[e]);
  return s.x + s.y;
}
__device__ __forceinline__ float dot(const float2 (&u)[8], const float2 (&v)[8]) {
  float2 s = mul(u[0], v[0]);
#pragma unroll
  for (int e = 1; e < 8; ++e) s = fma(u[e], v[e], s);
  return s.x + s.y;
}

// f becomes xhat; returns 1 / deviation. Lanes past the head's end hold 0 and keep it.
template <int LPH>
__device__ __forceinline__ float normed(float2 (&f)[8], int kind, float per, float eps, bool ok) {
  if (kind == SWIN_NORM_LAYER) {
    const float mean = head_sum<LPH>(total(f)) * per;
    const float2 m = both(ok ? -mean : 0.f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = add(f[e], m);
  }
  const float rstd = rsqrtf(fmaf(head_sum<LPH>(dot(f, f)), per, eps));
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = mul(f[e], both(rstd));
  return rstd;
}

// A lane's 16 values of an item: two vectors, `second` bytes apart.
template <typename T>
struct Pair {
  Raw<T> a, b;
  __device__ __forceinline__ void load(const uint8_t *p, int second, bool wide, bool there) {
    a = b = Raw<T>{};
    if (there) {
      load8(p, a, wide);
      load8(p + second, b, wide);
    }
  }
  __device__ __forceinline__ void unpack_to(float2 (&f)[8]) const {
    float2 x[4], y[4];
    unpack(a, x);
    unpack(b, y);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = x[e], f[e + 4] = y[e];
  }
  __device__ __forceinline__ void store(const float2 (&f)[8], uint8_t *p, int second, bool wide) {
    float2 x[4], y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = f[e], y[e] = f[e + 4];
    pack(x, a);
    pack(y, b);
    store8(p, 0, a, wide);
    store8(p, second, b, wide);
  }
};

// A CTA works on tiles of one part: all heads of some consecutive tokens, so that
// its lanes read and write whole runs of a row. LPH lanes hold a head (as many as a
// power of two needs; those past the head idle), 16 values each, in two vectors
// whose values turn with one another: half a rotary apart, so that no value leaves
// its lane (with one vector a lane and eight shuffles: 138 240 x 2 x 8 heads of 128
// 413 us). A token's cosines and sines serve all heads of the tile from shared
// memory. The next tile's loads are in flight while a tile is worked on; its table
// is one of two, so that a tile needs one barrier.
template <typename T, int LPH, bool kBwd, bool kNorm, bool kBeta>
__global__ void __launch_bounds__(threads_of(kBwd), kBlocks)
    heads_kernel(const __grid_constant__ Args a) {
  constexpr int kThreads = threads_of(kBwd), U = items_of(sizeof(T)), kGroups = kThreads / LPH,
                kItems = kGroups * U;
  extern __shared__ __align__(16) float smem[];
  int pi = 0;
#pragma unroll
  for (int i = 1; i < SWIN_HEAD_PARTS_MAX; ++i)
    if (i < a.count && (int)blockIdx.x >= a.parts[i].cta0) pi = i;
  const Part &p = a.parts[pi];
  const int cta = blockIdx.x - p.cta0, chunk = cta % p.chunks;
  const int group = threadIdx.x / LPH, v = threadIdx.x % LPH;
  const int rot16 = p.rot >> 4, kind = kNorm ? p.kind : SWIN_NORM_NONE;
  const bool ok = v * 16 < a.hd, turns = v < rot16;
  const float per = 1.f / (float)a.hd;
  // a lane's vectors: v and v + rot16 of those that turn, two neighbours of the others
  const int vec_a = turns ? v : 2 * v, vec_b = turns ? v + rot16 : 2 * v + 1;
  const int second = (vec_b - vec_a) * vec_bytes<T>();
  float2 gamma[8], beta[8], dgamma[8], dbeta[8];
  float4 *const held = reinterpret_cast<float4 *>(smem) + v;  // backward: gamma's quads, LPH apart
  if (kNorm) {
    float2 x[4], y[4];
    load_param(p.gamma, vec_a, ok, 1.f, x);
    load_param(p.gamma, vec_b, ok, 1.f, y);
    if (kBwd) {
      if (group == 0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          held[j * LPH] = make_float4(x[2 * j].x, x[2 * j].y, x[2 * j + 1].x, x[2 * j + 1].y);
          held[(j + 2) * LPH] = make_float4(y[2 * j].x, y[2 * j].y, y[2 * j + 1].x, y[2 * j + 1].y);
        }
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) gamma[e] = x[e], gamma[e + 4] = y[e];
    }
    if (!kBwd && kBeta) {
      load_param(p.beta, vec_a, ok, 0.f, x);
      load_param(p.beta, vec_b, ok, 0.f, y);
#pragma unroll
      for (int e = 0; e < 4; ++e) beta[e] = x[e], beta[e + 4] = y[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) dgamma[e] = dbeta[e] = make_float2(0.f, 0.f);
  }
  // where this lane's items lie: the same in every tile
  const int heads = (int)p.by_heads.d, here = min(heads, p.heads - chunk * kItems);  // of a chunk, and of this one
  const uint32_t rows = (uint32_t)a.rows, row_step = (uint32_t)(p.tile_rows * (p.ctas / p.chunks));
  uint32_t t0 = (uint32_t)(p.tile_rows * (cta / p.chunks));
  int tl[U];
  bool some[U];
  const uint8_t *px[U], *pdy[kBwd ? U : 1];
  uint8_t *po[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int l = group + u * kGroups;
    tl[u] = (int)p.by_heads.div(l);
    const int head = l - tl[u] * heads;
    some[u] = ok && tl[u] < p.tile_rows && head < here;
    if (!some[u]) tl[u] = 0;
    const int64_t row = (int64_t)t0 + tl[u];
    const int64_t at = ((int64_t)(chunk * kItems + head) * a.hd + vec_a * 8) * (int)sizeof(T);
    px[u] = p.x + row * p.x_stride + at;
    if (kBwd) pdy[kBwd ? u : 0] = p.dy + row * p.dy_stride + at;
    po[u] = p.out + row * p.out_stride + at;
  }
  const int64_t x_step = (int64_t)row_step * p.x_stride, dy_step = (int64_t)row_step * p.dy_stride,
                out_step = (int64_t)row_step * p.out_stride;
  const bool reads_x = !kBwd || kind != SWIN_NORM_NONE;
  Filler filler;
  filler.init<kThreads>(a, p.rot);
  Pair<T> in[U], grad[kBwd ? U : 1];
  auto fetch = [&](uint32_t first) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool there = some[u] && first + tl[u] < rows;
      in[u].load(px[u], second, p.wide_x, there && reads_x);
      px[u] += x_step;
      if (kBwd) {
        grad[kBwd ? u : 0].load(pdy[kBwd ? u : 0], second, p.wide_dy, there);
        pdy[kBwd ? u : 0] += dy_step;
      }
    }
  };
  if (t0 < rows) fetch(t0);
  float *const tables = smem + (kBwd ? kParamFloats : 0), *table = tables;
  for (int copy = 0; t0 < rows; t0 += row_step, copy ^= 1) {
    Pair<T> in_now[U], grad_now[kBwd ? U : 1];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      in_now[u] = in[u];
      if (kBwd) grad_now[kBwd ? u : 0] = grad[kBwd ? u : 0];
    }
    if (t0 + row_step < rows) fetch(t0 + row_step);
    if (rot16) {
      table = tables + copy * a.table;
      filler.fill(a, rot16, t0, p.tile_rows, table);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool there = some[u] && t0 + tl[u] < rows;
      float2 f[8];
      const float *quads = table + tl[u] * table_row(rot16) + v * 4;
      if (!kBwd) {
        in_now[u].unpack_to(f);
        if (kNorm && kind != SWIN_NORM_NONE) {
          normed<LPH>(f, kind, per, p.eps, ok);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = kBeta ? fma(f[e], gamma[e], beta[e]) : mul(f[e], gamma[e]);
        }
        if (turns) turn(f, a.layout, quads, rot16);
      } else {
        grad_now[kBwd ? u : 0].unpack_to(f);
        if (turns) turn(f, a.layout, quads, rot16);
        if (kind != SWIN_NORM_NONE) {
          if (!there)  // its row of the table was never written
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = make_float2(0.f, 0.f);
          float2 hat[8];
          in_now[u].unpack_to(hat);
          const float rstd = normed<LPH>(hat, kind, per, p.eps, ok);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            dgamma[e] = fma(f[e], hat[e], dgamma[e]);
            if (kBeta) dbeta[e] = add(dbeta[e], f[e]);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 g = held[j * LPH];
            f[2 * j] = mul(f[2 * j], make_float2(g.x, g.y));
            f[2 * j + 1] = mul(f[2 * j + 1], make_float2(g.z, g.w));
          }
          const float mh = head_sum<LPH>(dot(f, hat)) * per;
          const float mg = kind == SWIN_NORM_LAYER ? head_sum<LPH>(total(f)) * per : 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            f[e] = mul(fma(hat[e], both(-mh), add(f[e], both(-mg))), both(rstd));
        }
      }
      if (there) in_now[u].store(f, po[u], second, p.wide_out);
      po[u] += out_step;
    }
  }
  if (kBwd && p.sums) {
    // the groups of a warp, then the warps, in a fixed order
    constexpr int kWidth = LPH * 16;  // floats of a warp's sums
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = 16; o >= LPH; o >>= 1) {
        dgamma[e] = add(dgamma[e], make_float2(__shfl_xor_sync(0xffffffffu, dgamma[e].x, o), __shfl_xor_sync(0xffffffffu, dgamma[e].y, o)));
        if (kBeta) dbeta[e] = add(dbeta[e], make_float2(__shfl_xor_sync(0xffffffffu, dbeta[e].x, o), __shfl_xor_sync(0xffffffffu, dbeta[e].y, o)));
      }
      const int c = (e < 4 ? vec_a : vec_b) * 8 + 2 * (e & 3);
      if (lane < LPH && ok) {
        float *buf = smem + warp * 2 * kWidth + c;
        buf[0] = dgamma[e].x;
        buf[1] = dgamma[e].y;
        buf[kWidth] = dbeta[e].x;
        buf[kWidth + 1] = dbeta[e].y;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.hd; i += kThreads) {
      const int which = i >= a.hd, c = i - which * a.hd;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) s += smem[(w * 2 + which) * kWidth + c];
      p.sums[((int64_t)cta * 2 + which) * a.hd + c] = s;
    }
  }
}

// Lanes of a head, a power of two.
inline int lanes_of(int hd) {
  int l = 1;
  while (l * 16 < hd) l *= 2;
  return l;
}

template <typename T, int LPH, bool kBwd, bool kNorm, bool kBeta>
int launch_kernel(const Args &a, int ctas, size_t smem, cudaStream_t st) {
  auto k = heads_kernel<T, LPH, kBwd, kNorm, kBeta>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SWIN_ERR_CUDA;
  k<<<ctas, threads_of(kBwd), smem, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

template <typename T, int LPH>
int launch_lanes(const Args &a, bool bwd, bool norm, bool beta, int ctas, size_t smem, cudaStream_t st) {
  if (bwd) return beta ? launch_kernel<T, LPH, true, true, true>(a, ctas, smem, st)
                       : launch_kernel<T, LPH, true, true, false>(a, ctas, smem, st);
  if (norm) return beta ? launch_kernel<T, LPH, false, true, true>(a, ctas, smem, st)
                        : launch_kernel<T, LPH, false, true, false>(a, ctas, smem, st);
  return launch_kernel<T, LPH, false, false, false>(a, ctas, smem, st);
}

// bwd: with a norm (a backward without one is a forward). beta: some part has one, or wants its gradient.
template <typename T>
int launch_heads(const Args &a, bool bwd, bool norm, bool beta, int ctas, size_t smem, cudaStream_t st) {
  switch (lanes_of(a.hd)) {
    case 1: return launch_lanes<T, 1>(a, bwd, norm, beta, ctas, smem, st);
    case 2: return launch_lanes<T, 2>(a, bwd, norm, beta, ctas, smem, st);
    case 4: return launch_lanes<T, 4>(a, bwd, norm, beta, ctas, smem, st);
    case 8: return launch_lanes<T, 8>(a, bwd, norm, beta, ctas, smem, st);
    default: return launch_lanes<T, 16>(a, bwd, norm, beta, ctas, smem, st);
  }
}

// The kernel of either type (swin_heads_bf16.cu, swin_heads_f32.cu).
int launch_bf16(const Args &a, bool bwd, bool norm, bool beta, int ctas, size_t smem, cudaStream_t st);
int launch_f32(const Args &a, bool bwd, bool norm, bool beta, int ctas, size_t smem, cudaStream_t st);

}  // namespace heads
}  // namespace swin
