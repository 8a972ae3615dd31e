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

constexpr int kThreads = 256;
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
  FastDiv by_heads;
  float eps;
  const float *gamma, *beta;
  float *sums, *dgamma, *dbeta;  // sums: [ctas][2][hd], or NULL
  int cta0, ctas;
  bool wide_x, wide_dy, wide_out;  // fp32: 32-byte pieces
};

struct Args {
  int rows, hd, ndim, count, layout;
  int table;  // cosines and sines (pairs of floats) of one of a tile's two tables
  FastDiv by_tokens, by_pairs, stride[3], extent[3];
  float amplitude;
  const void *positions;
  int position_bits, shared;
  Part parts[SWIN_HEAD_PARTS_MAX];
  uint64_t freq[kMaxPairs];
  uint8_t axis[kMaxPairs];
};

// Items (a head of a token) a thread takes at a time: all are asked for before any is worked on.
constexpr int items_of(bool bwd, int bytes) { return bwd ? 2 : bytes == 2 ? 4 : 2; }
// Resident CTAs an SM: what the launch bound asks for.
constexpr int blocks_of(bool bwd) { return bwd ? 2 : 4; }

// Cosines and sines of `tokens` rows from row t0 on, times the amplitude: [token][pair].
__device__ __forceinline__ void fill_table(const Args &a, int rot, int64_t t0, int tokens, float2 *table) {
  const int pairs = rot >> 1;
  for (int e = threadIdx.x; e < tokens * pairs; e += kThreads) {
    const int t = (int)a.by_pairs.div(e), pair = e - t * pairs;
    const int64_t row = t0 + t;
    if (row >= a.rows) break;
    const int axis = a.axis[pair];
    const uint32_t tok = (uint32_t)row - a.by_tokens.div((uint32_t)row) * a.by_tokens.d;
    int64_t at;
    if (a.position_bits == 0) {
      const uint32_t c = a.stride[axis].div(tok);
      at = c - a.extent[axis].div(c) * a.extent[axis].d;
    } else {
      const int64_t i = (a.shared ? (int64_t)tok : row) * a.ndim + axis;
      at = a.position_bits == 64 ? static_cast<const int64_t *>(a.positions)[i]
                                 : (int64_t) static_cast<const int32_t *>(a.positions)[i];
    }
    // the fraction of a turn, of which 32 bits are kept: half turns from -1 to 1
    const uint64_t turn = (uint64_t)at * a.freq[pair];
    const float half_turns = (float)(int32_t)(uint32_t)(turn >> 32) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    table[e] = make_float2(c * a.amplitude, s * a.amplitude);
  }
}

// Turns a head's vector `v` (of the LPH that its lanes hold) by the table's row of its token.
template <int LPH>
__device__ __forceinline__ void turn(float2 (&f)[4], int v, int rot8, int layout, const float2 *row) {
  if (layout == SWIN_ROTARY_HALF) {
    const int half8 = rot8 >> 1;
    const bool low = v < half8;
    const int from = low ? v + half8 : v < rot8 ? v - half8 : v;
    float2 q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      q[e] = make_float2(__shfl_sync(0xffffffffu, f[e].x, from, LPH), __shfl_sync(0xffffffffu, f[e].y, from, LPH));
    if (v >= rot8) return;
    const float4 *cs = reinterpret_cast<const float4 *>(row + 8 * (low ? v : v - half8));
    const float sign = low ? -1.f : 1.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4 k = cs[e];  // cos, sin of two pairs
      f[e] = fma(f[e], make_float2(k.x, k.z), mul(q[e], make_float2(sign * k.y, sign * k.w)));
    }
  } else {
    if (v >= rot8) return;
    const float4 *cs = reinterpret_cast<const float4 *>(row + 4 * v);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float4 k = cs[e >> 1];
      f[e] = make_float2(fmaf(f[e].x, k.x, -f[e].y * k.y), fmaf(f[e].x, k.y, f[e].y * k.x));
      f[e + 1] = make_float2(fmaf(f[e + 1].x, k.z, -f[e + 1].y * k.w), fmaf(f[e + 1].x, k.w, f[e + 1].y * k.z));
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

__device__ __forceinline__ float total(const float2 (&u)[4]) {
  const float2 s = add(add(u[0], u[1]), add(u[2], u[3]));
  return s.x + s.y;
}
__device__ __forceinline__ float dot(const float2 (&u)[4], const float2 (&v)[4]) {
  float2 s = mul(u[0], v[0]);
#pragma unroll
  for (int e = 1; e < 4; ++e) s = fma(u[e], v[e], s);
  return s.x + s.y;
}

// f becomes xhat; returns 1 / deviation. Vectors past the head's end are and stay 0.
template <int LPH>
__device__ __forceinline__ float normed(float2 (&f)[4], int kind, float per, float eps, bool ok) {
  if (kind == SWIN_NORM_LAYER) {
    const float mean = head_sum<LPH>(total(f)) * per;
    const float2 m = both(ok ? -mean : 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = add(f[e], m);
  }
  const float rstd = 1.f / sqrtf(fmaf(head_sum<LPH>(dot(f, f)), per, eps));
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = mul(f[e], both(rstd));
  return rstd;
}

// A CTA works on tiles of one part: consecutive heads of consecutive tokens, so
// that its lanes read and write whole runs of a row. LPH lanes hold a head, eight
// values each (as many lanes as a power of two needs; those past the head idle).
// A token's cosines and sines serve all heads of its tile from shared memory; they
// are worked out while the tile's loads are in flight, into one of two tables, so a
// tile needs one barrier.
template <typename T, int LPH, bool kBwd, bool kNorm>
__global__ void __launch_bounds__(kThreads, blocks_of(kBwd)) heads_kernel(const __grid_constant__ Args a) {
  constexpr int U = items_of(kBwd, sizeof(T)), kGroups = kThreads / LPH, kItems = kGroups * U;
  extern __shared__ __align__(16) float2 smem[];
  int pi = 0;
#pragma unroll
  for (int i = 1; i < SWIN_HEAD_PARTS_MAX; ++i)
    if (i < a.count && (int)blockIdx.x >= a.parts[i].cta0) pi = i;
  const Part &p = a.parts[pi];
  const int cta = blockIdx.x - p.cta0;
  const int group = threadIdx.x / LPH, v = threadIdx.x % LPH;
  const bool ok = v * 8 < a.hd;
  const int heads = p.heads, rot8 = p.rot >> 3, kind = kNorm ? p.kind : SWIN_NORM_NONE;
  const float per = 1.f / (float)a.hd;
  const uint32_t head_bytes = a.hd * sizeof(T), lane_bytes = v * vec_bytes<T>();
  float2 gamma[4], beta[4], dgamma[4], dbeta[4];
  if (kNorm) {
    load_param(p.gamma, v, ok, 1.f, gamma);
    if (!kBwd) load_param(p.beta, v, ok, 0.f, beta);
#pragma unroll
    for (int e = 0; e < 4; ++e) dgamma[e] = dbeta[e] = make_float2(0.f, 0.f);
  }
  // the tile's first item: head h0 of row t0
  const int64_t first = (int64_t)cta * kItems, step = (int64_t)p.ctas * kItems;
  int64_t t0 = first / heads, dt = step / heads;
  int h0 = (int)(first - t0 * heads), dh = (int)(step - dt * heads);
  int copy = 0;
  for (; t0 < a.rows; copy ^= 1) {
    Raw<T> in[U], grad[kBwd ? U : 1];
    int64_t row[U];
    int tl[U], head[U];
    bool there[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int l = h0 + group + u * kGroups;
      tl[u] = (int)p.by_heads.div(l);
      head[u] = l - tl[u] * heads;
      row[u] = t0 + tl[u];
      there[u] = ok && row[u] < a.rows;
      in[u] = Raw<T>{};
      if (kBwd) grad[kBwd ? u : 0] = Raw<T>{};
      if (there[u]) {
        const int64_t at = (int64_t)head[u] * head_bytes + lane_bytes;
        if (!kBwd || kind != SWIN_NORM_NONE) load8(p.x + row[u] * p.x_stride + at, in[u], p.wide_x);
        if (kBwd) load8(p.dy + row[u] * p.dy_stride + at, grad[kBwd ? u : 0], p.wide_dy);
      }
    }
    float2 *table = smem + copy * a.table;
    if (p.rot) {
      const int span = (int)p.by_heads.div(h0 + kItems - 1) + 1;
      fill_table(a, p.rot, t0, span, table);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float2 f[4];
      Raw<T> out;
      const float2 *cs = table + tl[u] * (p.rot >> 1);
      if (!kBwd) {
        unpack(in[u], f);
        if (kNorm && kind != SWIN_NORM_NONE) {
          normed<LPH>(f, kind, per, p.eps, ok);
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = fma(f[e], gamma[e], beta[e]);
        }
        if (p.rot) turn<LPH>(f, v, rot8, a.layout, cs);
      } else {
        unpack(grad[kBwd ? u : 0], f);
        if (p.rot) turn<LPH>(f, v, rot8, a.layout, cs);
        if (kind != SWIN_NORM_NONE) {
          if (!there[u])  // its row of the table was never written
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = make_float2(0.f, 0.f);
          float2 hat[4];
          unpack(in[u], hat);
          const float rstd = normed<LPH>(hat, kind, per, p.eps, ok);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            dgamma[e] = fma(f[e], hat[e], dgamma[e]);
            dbeta[e] = add(dbeta[e], f[e]);
            f[e] = mul(f[e], gamma[e]);
          }
          const float mh = head_sum<LPH>(dot(f, hat)) * per;
          const float mg = kind == SWIN_NORM_LAYER ? head_sum<LPH>(total(f)) * per : 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            f[e] = mul(fma(hat[e], both(-mh), add(f[e], both(-mg))), both(rstd));
        }
      }
      pack(f, out);
      if (there[u])
        store8(p.out, row[u] * p.out_stride + (int64_t)head[u] * head_bytes + lane_bytes, out, p.wide_out);
    }
    t0 += dt;
    h0 += dh;
    if (h0 >= heads) {
      h0 -= heads;
      ++t0;
    }
  }
  if (kBwd && p.sums) {
    // the groups of a warp, then the warps, in a fixed order
    float2 *buf = smem;  // [warp][2][LPH * 4] pairs
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int o = 16; o >= LPH; o >>= 1) {
        dgamma[e] = add(dgamma[e], make_float2(__shfl_xor_sync(0xffffffffu, dgamma[e].x, o), __shfl_xor_sync(0xffffffffu, dgamma[e].y, o)));
        dbeta[e] = add(dbeta[e], make_float2(__shfl_xor_sync(0xffffffffu, dbeta[e].x, o), __shfl_xor_sync(0xffffffffu, dbeta[e].y, o)));
      }
    }
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) < LPH) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        buf[(warp * 2 + 0) * LPH * 4 + v * 4 + e] = dgamma[e];
        buf[(warp * 2 + 1) * LPH * 4 + v * 4 + e] = dbeta[e];
      }
    }
    __syncthreads();
    const float *flat = reinterpret_cast<const float *>(buf);
    for (int i = threadIdx.x; i < 2 * a.hd; i += kThreads) {
      const int which = i >= a.hd, c = i - which * a.hd;
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) s += flat[(w * 2 + which) * LPH * 8 + c];
      p.sums[((int64_t)cta * 2 + which) * a.hd + c] = s;
    }
  }
}

// Lanes of a head, a power of two of at least two.
inline int lanes_of(int hd) {
  int l = 2;
  while (l * 8 < hd) l *= 2;
  return l;
}

template <typename T, int LPH, bool kBwd, bool kNorm>
int launch_kernel(const Args &a, int ctas, size_t smem, cudaStream_t st) {
  auto k = heads_kernel<T, LPH, kBwd, kNorm>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return SWIN_ERR_CUDA;
  k<<<ctas, kThreads, smem, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

template <typename T, int LPH>
int launch_lanes(const Args &a, bool bwd, bool norm, int ctas, size_t smem, cudaStream_t st) {
  if (bwd) return launch_kernel<T, LPH, true, true>(a, ctas, smem, st);
  if (norm) return launch_kernel<T, LPH, false, true>(a, ctas, smem, st);
  return launch_kernel<T, LPH, false, false>(a, ctas, smem, st);
}

template <typename T>
int launch_heads(const Args &a, bool bwd, bool norm, int ctas, size_t smem, cudaStream_t st) {
  switch (lanes_of(a.hd)) {
    case 2: return launch_lanes<T, 2>(a, bwd, norm, ctas, smem, st);
    case 4: return launch_lanes<T, 4>(a, bwd, norm, ctas, smem, st);
    case 8: return launch_lanes<T, 8>(a, bwd, norm, ctas, smem, st);
    case 16: return launch_lanes<T, 16>(a, bwd, norm, ctas, smem, st);
    default: return launch_lanes<T, 32>(a, bwd, norm, ctas, smem, st);
  }
}

// The kernel of either type (swin_heads_bf16.cu, swin_heads_f32.cu).
int launch_bf16(const Args &a, bool bwd, bool norm, int ctas, size_t smem, cudaStream_t st);
int launch_f32(const Args &a, bool bwd, bool norm, int ctas, size_t smem, cudaStream_t st);

}  // namespace heads
}  // namespace swin
