// swin_rows.cu -- the operators around the attention of a block, on rows of C
// channels (tokens of [B, grid..., C]): the norm before the block, the
// residual join after it, and dropout; forward and backward (sm_103a).
//
//   norm   h = N(x);                    N: LayerNorm or RMSNorm, gamma, beta
//   join   y = x + scale * gate * path * D(N_post(z)),   h = N_pre(y)
//
// xhat = (x - mean) rstd (RMSNorm: mean = 0), N = xhat gamma + beta. With
// g = dh gamma: N^T dh = rstd (g - m(g) - xhat m(g xhat)), m the mean over the
// row (no m(g) term for RMSNorm). Join backward, from the stored y:
//   dx = dy' = dy + N_pre^T dh,  G = keep/kept * path * dy',
//   dz = N_post^T (scale gate gamma_post G),
//   S1 = sum over an image's rows of G zhat (G z without a post norm), S0 = of G:
// every gradient of scale, gate, gamma_post and beta_post is S1 and S0 times
// per-channel factors, so the kernel carries two sums per channel for all four.
//
// What bounds them: HBM. Each is one pass: a row is read once into registers,
// its statistics are taken there (mean first, then centred squares: no
// cancellation when the mean is large), and the results leave as 16-byte
// stores. The statistics are recomputed by the backward instead of stored.
// A row belongs to TPR threads, each holding NV vectors of 8 channels; the
// channels of a thread never change, so gamma, beta, scale and gate stay in
// registers and the column sums (the parameter gradients) accumulate there,
// per CTA, and are folded in a fixed order by a second kernel: no atomics, the
// same bits every run. All sums and statistics are fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "swin_common.cuh"
#include "swin_philox.cuh"

namespace swin {
namespace {

struct Norm {
  int kind;
  float eps;
  const float *gamma, *beta;
};

struct RowArgs {
  int64_t rows, tokens, chunk;  // all rows; rows of one image; rows of one CTA
  int images, C;
  const void *x, *z;    // x: forward the residual stream (norm: its input), backward the stored y
  const void *dy, *dh;  // backward
  void *y, *h;          // forward
  void *dx, *dz;        // backward
  Norm post, pre;
  const float *scale, *gate;
  Drop drop, path;
  float *part_pre, *part_post;  // column sums [ctas][2][C], [slots][2][C]; NULL: not wanted
};

// ---- eight channels of a row -----------------------------------------------
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 v;
};
template <>
struct Raw<float> {
  float4 a, b;
};

template <typename T>
__device__ __forceinline__ Raw<T> load8(const void *base, int64_t vec);
template <>
__device__ __forceinline__ Raw<__nv_bfloat16> load8<__nv_bfloat16>(const void *base, int64_t vec) {
  return {static_cast<const uint4 *>(base)[vec]};
}
template <>
__device__ __forceinline__ Raw<float> load8<float>(const void *base, int64_t vec) {
  const float4 *p = static_cast<const float4 *>(base) + 2 * vec;
  return {p[0], p[1]};
}

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16> &r, float (&f)[8]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void unpack(const Raw<float> &r, float (&f)[8]) {
  f[0] = r.a.x, f[1] = r.a.y, f[2] = r.a.z, f[3] = r.a.w;
  f[4] = r.b.x, f[5] = r.b.y, f[6] = r.b.z, f[7] = r.b.w;
}

__device__ __forceinline__ void pack(const float (&f)[8], Raw<__nv_bfloat16> &r) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t *>(&h);
  }
  r.v = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float (&f)[8], Raw<float> &r) {
  r.a = make_float4(f[0], f[1], f[2], f[3]);
  r.b = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ void store8(void *base, int64_t vec, const Raw<__nv_bfloat16> &r) {
  static_cast<uint4 *>(base)[vec] = r.v;
}
__device__ __forceinline__ void store8(void *base, int64_t vec, const Raw<float> &r) {
  float4 *p = static_cast<float4 *>(base) + 2 * vec;
  p[0] = r.a;
  p[1] = r.b;
}

// Per-channel fp32 parameters of this thread's channels (absent: `none`).
__device__ __forceinline__ void load_param(const float *p, int vec, bool ok, float none, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = p && ok ? __ldg(p + 8 * vec + e) : none;
}

// ---- sums over a row ---------------------------------------------------------
// K sums over the TPR threads of a row. Rows of up to 32 threads stay inside a
// warp; wider rows are the whole CTA and exchange one value per warp through
// one of two shared buffers (used in turn: one barrier per sum).
template <int TPR, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float *xchg, int &turn) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float *buf = xchg + turn * (2 * W);
    turn ^= 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) buf[k * W + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += buf[k * W + w];
      v[k] = s;
    }
  }
}

constexpr int block_of(int tpr) { return tpr > 32 ? tpr : 256; }

// Mean and 1 / deviation of up to two rows at once (u with norm kind ku, v
// with kv; kind NONE leaves that row alone). inv = 1 / C.
template <int TPR, int NV, int K>
__device__ __forceinline__ void row_stats(const float (&u)[K][NV][8], const bool (&ok)[NV], const int (&kind)[K],
                                          const float (&eps)[K], float inv, float (&mean)[K], float (&rstd)[K],
                                          float *xchg, int &turn) {
  bool any_mean = false;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    mean[k] = 0.f;
    any_mean = any_mean || kind[k] == SWIN_NORM_LAYER;
  }
  if (any_mean) {
    float s[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      s[k] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s[k] += u[k][j][e];
    }
    row_sum<TPR, K>(s, xchg, turn);
#pragma unroll
    for (int k = 0; k < K; ++k) mean[k] = kind[k] == SWIN_NORM_LAYER ? s[k] * inv : 0.f;
  }
  float q[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    q[k] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = ok[j] ? u[k][j][e] - mean[k] : 0.f;
        q[k] = fmaf(d, d, q[k]);
      }
  }
  row_sum<TPR, K>(q, xchg, turn);
#pragma unroll
  for (int k = 0; k < K; ++k) rstd[k] = 1.0f / sqrtf(fmaf(q[k], inv, eps[k]));
}

// ---- forward -----------------------------------------------------------------
template <typename T, int TPR, int NV, bool kBranch, bool kPre>
__global__ void __launch_bounds__(block_of(TPR)) rows_fwd_kernel(const RowArgs a) {
  constexpr int kThreads = block_of(TPR), kWarps = kThreads / 32;
  constexpr int RPW = TPR < 32 ? 32 / TPR : 1;  // rows a warp works on at once
  __shared__ float xchg[TPR > 32 ? 4 * (TPR / 32) : 1];
  int turn = 0;
  const int lane = TPR > 32 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  const int C8 = a.C >> 3;
  const float inv = 1.0f / (float)a.C;
  bool ok[NV];
  float gpre[NV][8], bpre[NV][8], wg[NV][8], wb[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    ok[j] = j * TPR + lane < C8;
    if constexpr (kPre) {
      load_param(a.pre.gamma, j * TPR + lane, ok[j], 1.f, gpre[j]);
      load_param(a.pre.beta, j * TPR + lane, ok[j], 0.f, bpre[j]);
    }
  }
  Philox ph;
  ph.init(a.drop);
  const bool post = a.post.kind != SWIN_NORM_NONE;

  const int64_t L = (int64_t)blockIdx.x * a.chunk;
  const int64_t R = min(L + a.chunk, a.rows);
  const int64_t stride = TPR > 32 ? 1 : (int64_t)kWarps * RPW;
  const int64_t first = TPR > 32 ? 0 : (threadIdx.x >> 5) * RPW;
  const int sub = TPR < 32 ? (threadIdx.x & 31) / TPR : 0;
  // one image of the CTA's rows at a time: the gate and the path decision change with it
  for (int64_t s = L; s < R;) {
    const int64_t b = s / a.tokens;
    const int64_t e1 = min(R, (b + 1) * a.tokens);
    if constexpr (kBranch) {
      float path = a.drop.thr ? a.drop.scale : 1.f;
      if (a.path.thr) {
        Philox pp;
        pp.init(a.path);
        path = keep_one(pp, (uint64_t)b, a.path.thr) ? path * a.path.scale : 0.f;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float t[8];
        load_param(a.scale, j * TPR + lane, ok[j], 1.f, wg[j]);
        load_param(a.gate ? a.gate + b * a.C : nullptr, j * TPR + lane, ok[j], 1.f, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) wb[j][e] = wg[j][e] = wg[j][e] * t[e] * path;
        load_param(a.post.gamma, j * TPR + lane, ok[j] && post, 1.f, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) wg[j][e] *= t[e];
        load_param(a.post.beta, j * TPR + lane, ok[j] && post, 0.f, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) wb[j][e] *= t[e];
      }
    }
    for (int64_t r0 = s + first; r0 < e1; r0 += stride) {
      const int64_t row = r0 + sub;
      const bool live = row < e1;
      const int64_t vec0 = row * C8 + lane;
      float v[1][NV][8], u[1][NV][8];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Raw<T> rx = {}, rz = {};
        if (ok[j] && live) {
          rx = load8<T>(a.x, vec0 + j * TPR);
          if constexpr (kBranch) rz = load8<T>(a.z, vec0 + j * TPR);
        }
        unpack(rx, v[0][j]);
        unpack(rz, u[0][j]);
      }
      if constexpr (kBranch) {
        float mean[1] = {0.f}, rstd[1] = {1.f};
        if (post) row_stats<TPR, NV, 1>(u, ok, {a.post.kind}, {a.post.eps}, inv, mean, rstd, xchg, turn);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          uint4 bits = make_uint4(~0u, ~0u, ~0u, ~0u);
          if (a.drop.thr) bits = ph.block((uint64_t)(vec0 + j * TPR));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float hat = post ? (u[0][j][e] - mean[0]) * rstd[0] : u[0][j][e];
            const float br = fmaf(hat, wg[j][e], wb[j][e]);
            v[0][j][e] += keep_of(bits, e, a.drop.thr) ? br : 0.f;
          }
          Raw<T> out;
          pack(v[0][j], out);
          if (ok[j] && live) store8(a.y, vec0 + j * TPR, out);
          unpack(out, v[0][j]);  // h is the norm of y as stored
        }
      }
      if constexpr (kPre) {
        float mean[1], rstd[1];
        row_stats<TPR, NV, 1>(v, ok, {a.pre.kind}, {a.pre.eps}, inv, mean, rstd, xchg, turn);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = fmaf((v[0][j][e] - mean[0]) * rstd[0], gpre[j][e], bpre[j][e]);
          Raw<T> out;
          pack(o, out);
          if (ok[j] && live) store8(a.h, vec0 + j * TPR, out);
        }
      }
    }
    s = e1;
  }
}

// ---- backward ----------------------------------------------------------------
// Sums the CTA's copies of this thread's channels and writes them: dst[C].
template <int TPR, int NV>
__device__ __forceinline__ void flush(float (&acc)[NV][8], float *dst, int C8, float *buf) {
  constexpr int kThreads = block_of(TPR);
  const int lane = TPR > 32 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  if constexpr (TPR > 32) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int v = j * TPR + lane;
      if (v < C8) {
        float4 *p = reinterpret_cast<float4 *>(dst + 8 * v);
        p[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
        p[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
      }
    }
  } else {
    constexpr int G = kThreads / TPR, W = TPR * NV * 8;  // rows in flight, channels of a row (padded)
    const int g = threadIdx.x / TPR;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float4 *p = reinterpret_cast<float4 *>(buf + g * W + 8 * (j * TPR + lane));
      p[0] = make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      p[1] = make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 8 * C8; c += kThreads) {
      float s = 0.f;
#pragma unroll 8
      for (int k = 0; k < G; ++k) s += buf[k * W + c];
      dst[c] = s;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[j][e] = 0.f;
}

template <typename T, int TPR, int NV, bool kBranch, bool kPre>
__global__ void __launch_bounds__(block_of(TPR)) rows_bwd_kernel(const RowArgs a) {
  constexpr int kThreads = block_of(TPR), kWarps = kThreads / 32;
  constexpr int RPW = TPR < 32 ? 32 / TPR : 1;
  constexpr int K = (kBranch ? 1 : 0) + (kPre ? 1 : 0);  // rows with statistics
  constexpr int kZ = 0, kY = kBranch ? 1 : 0;            // their indexes
  __shared__ float xchg[TPR > 32 ? 4 * (TPR / 32) : 1];
  __shared__ __align__(16) float buf[TPR > 32 ? 4 : kThreads * NV * 8];
  int turn = 0;
  const int lane = TPR > 32 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  const int C8 = a.C >> 3;
  const float inv = 1.0f / (float)a.C;
  bool ok[NV];
  float gpre[NV][8], w[NV][8];
  float a1[NV][8], a0[NV][8], b1[NV][8], b0[NV][8];  // column sums: dh yhat, dh; G zhat, G
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    ok[j] = j * TPR + lane < C8;
    if constexpr (kPre) load_param(a.pre.gamma, j * TPR + lane, ok[j], 1.f, gpre[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) a1[j][e] = a0[j][e] = b1[j][e] = b0[j][e] = 0.f;
  }
  Philox ph;
  ph.init(a.drop);
  const bool post = a.post.kind != SWIN_NORM_NONE;

  const int64_t L = (int64_t)blockIdx.x * a.chunk;
  const int64_t R = min(L + a.chunk, a.rows);
  const int64_t stride = TPR > 32 ? 1 : (int64_t)kWarps * RPW;
  const int64_t first = TPR > 32 ? 0 : (threadIdx.x >> 5) * RPW;
  const int sub = TPR < 32 ? (threadIdx.x & 31) / TPR : 0;
  for (int64_t s = L; s < R;) {
    const int64_t b = s / a.tokens;
    const int64_t e1 = min(R, (b + 1) * a.tokens);
    float path = 1.f;  // kept values' scale times the image's path factor
    if constexpr (kBranch) {
      path = a.drop.thr ? a.drop.scale : 1.f;
      if (a.path.thr) {
        Philox pp;
        pp.init(a.path);
        path = keep_one(pp, (uint64_t)b, a.path.thr) ? path * a.path.scale : 0.f;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float t[8];
        load_param(a.scale, j * TPR + lane, ok[j], 1.f, w[j]);
        load_param(a.gate ? a.gate + b * a.C : nullptr, j * TPR + lane, ok[j], 1.f, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[j][e] *= t[e];
        load_param(a.post.gamma, j * TPR + lane, ok[j] && post, 1.f, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) w[j][e] *= t[e];
      }
    }
    for (int64_t r0 = s + first; r0 < e1; r0 += stride) {
      const int64_t row = r0 + sub;
      const bool live = row < e1;
      const int64_t vec0 = row * C8 + lane;
      float u[K][NV][8], g[NV][8], dh[NV][8];  // z and y rows; dy; dh
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Raw<T> ry = {}, rz = {}, rg = {}, rh = {};
        if (ok[j] && live) {
          if constexpr (kPre) {
            ry = load8<T>(a.x, vec0 + j * TPR);
            if (a.dh) rh = load8<T>(a.dh, vec0 + j * TPR);
          }
          if constexpr (kBranch)
            if (a.z) rz = load8<T>(a.z, vec0 + j * TPR);
          if (a.dy) rg = load8<T>(a.dy, vec0 + j * TPR);
        }
        if constexpr (kBranch) unpack(rz, u[kZ][j]);
        if constexpr (kPre) unpack(ry, u[kY][j]);
        unpack(rg, g[j]);
        unpack(rh, dh[j]);
      }
      float mean[K], rstd[K];
      int kind[K];
      float eps[K];
      if constexpr (kBranch) kind[kZ] = a.post.kind, eps[kZ] = post ? a.post.eps : 1.f;
      if constexpr (kPre) kind[kY] = a.pre.kind, eps[kY] = a.pre.eps;
      if (kPre || post)
        row_stats<TPR, NV, K>(u, ok, kind, eps, inv, mean, rstd, xchg, turn);
      if constexpr (kPre) {
        float c[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float hat = ok[j] ? (u[kY][j][e] - mean[kY]) * rstd[kY] : 0.f;
            u[kY][j][e] = hat;
            a1[j][e] = fmaf(dh[j][e], live ? hat : 0.f, a1[j][e]);
            a0[j][e] += dh[j][e];
            dh[j][e] *= gpre[j][e];
            c[0] += dh[j][e];
            c[1] = fmaf(dh[j][e], hat, c[1]);
          }
        row_sum<TPR, 2>(c, xchg, turn);
        const float c0 = a.pre.kind == SWIN_NORM_LAYER ? c[0] * inv : 0.f, c1 = c[1] * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            g[j][e] = fmaf(rstd[kY], dh[j][e] - fmaf(u[kY][j][e], c1, c0), g[j][e]);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Raw<T> out;
        pack(g[j], out);
        if (ok[j] && live) store8(a.dx, vec0 + j * TPR, out);
      }
      if constexpr (kBranch) {
        float c[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          uint4 bits = make_uint4(~0u, ~0u, ~0u, ~0u);
          if (a.drop.thr) bits = ph.block((uint64_t)(vec0 + j * TPR));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float gd = keep_of(bits, e, a.drop.thr) && ok[j] && live ? g[j][e] * path : 0.f;
            const float hat = !ok[j] || !live ? 0.f : post ? (u[kZ][j][e] - mean[kZ]) * rstd[kZ] : u[kZ][j][e];
            u[kZ][j][e] = hat;
            b1[j][e] = fmaf(gd, hat, b1[j][e]);
            b0[j][e] += gd;
            g[j][e] = gd * w[j][e];
            c[0] += g[j][e];
            c[1] = fmaf(g[j][e], hat, c[1]);
          }
        }
        if (post) {
          row_sum<TPR, 2>(c, xchg, turn);
          const float c0 = a.post.kind == SWIN_NORM_LAYER ? c[0] * inv : 0.f, c1 = c[1] * inv;
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) g[j][e] = rstd[kZ] * (g[j][e] - fmaf(u[kZ][j][e], c1, c0));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          Raw<T> out;
          pack(g[j], out);
          if (ok[j] && live) store8(a.dz, vec0 + j * TPR, out);
        }
      }
    }
    // with a gate the sums are kept per image: slot CTA + image (a CTA's next
    // image takes its next slot, the next CTA's first is one further)
    if constexpr (kBranch)
      if (a.part_post && (a.gate || e1 == R)) {
        float *dst = a.part_post + ((int64_t)blockIdx.x + (a.gate ? b : 0)) * 2 * a.C;
        flush<TPR, NV>(b1, dst, C8, buf);
        flush<TPR, NV>(b0, dst + a.C, C8, buf);
      }
    s = e1;
  }
  if constexpr (kPre)
    if (a.part_pre) {
      float *dst = a.part_pre + (int64_t)blockIdx.x * 2 * a.C;
      flush<TPR, NV>(a1, dst, C8, buf);
      flush<TPR, NV>(a0, dst + a.C, C8, buf);
    }
}

// ---- parameter gradients from the column sums ----------------------------------
struct ColArgs {
  int64_t tokens, chunk, rows;
  int images, C, ctas;
  bool post_norm;
  const float *part_pre, *part_post;
  const float *scale, *gate, *gamma, *beta;  // gamma, beta: the post norm's
  float *dpre_gamma, *dpre_beta, *dpost_gamma, *dpost_beta, *dscale, *dgate;
};

constexpr int kColLanes = 16;

// Sum over the lanes of a block (32 channels x kColLanes), in lane order.
__device__ __forceinline__ float lane_sum(float v, float *buf) {
  __syncthreads();
  buf[threadIdx.y * 32 + threadIdx.x] = v;
  __syncthreads();
  float s = 0.f;
  if (threadIdx.y == 0)
#pragma unroll
    for (int k = 0; k < kColLanes; ++k) s += buf[k * 32 + threadIdx.x];
  return s;
}

// Block (tile, 0): the sums over all rows of 32 channels. Block (tile, 1 + b):
// image b's gate gradient.
__global__ void __launch_bounds__(32 * kColLanes) columns_kernel(const ColArgs a) {
  __shared__ float buf[32 * kColLanes];
  const int tiles = (a.C + 31) / 32;
  const int tile = (int)(blockIdx.x % tiles);
  const int64_t task = blockIdx.x / tiles;
  const int c = tile * 32 + threadIdx.x, cc = min(c, a.C - 1);
  const bool own = threadIdx.y == 0 && c < a.C;
  const int64_t C2 = 2 * (int64_t)a.C;
  if (task > 0) {
    const int64_t b = task - 1;
    const int64_t s0 = a.tokens * b / a.chunk + b, s1 = (a.tokens * (b + 1) - 1) / a.chunk + b;
    float v1 = 0.f, v0 = 0.f;
    if (a.rows)
      for (int64_t s = s0 + threadIdx.y; s <= s1; s += kColLanes) {
        v1 += a.part_post[s * C2 + cc];
        v0 += a.part_post[s * C2 + a.C + cc];
      }
    v1 = lane_sum(v1, buf);
    v0 = lane_sum(v0, buf);
    if (own) {
      const float gm = a.post_norm && a.gamma ? a.gamma[c] : 1.f, bt = a.post_norm && a.beta ? a.beta[c] : 0.f;
      a.dgate[b * a.C + c] = (a.scale ? a.scale[c] : 1.f) * fmaf(gm, v1, bt * v0);
    }
    return;
  }
  if (a.dpre_gamma || a.dpre_beta) {
    float v1 = 0.f, v0 = 0.f;
#pragma unroll 4
    for (int s = threadIdx.y; s < a.ctas; s += kColLanes) {
      v1 += a.part_pre[s * C2 + cc];
      v0 += a.part_pre[s * C2 + a.C + cc];
    }
    v1 = lane_sum(v1, buf);
    v0 = lane_sum(v0, buf);
    if (own && a.dpre_gamma) a.dpre_gamma[c] = v1;
    if (own && a.dpre_beta) a.dpre_beta[c] = v0;
  }
  if (a.dpost_gamma || a.dpost_beta || a.dscale) {
    float v1 = 0.f, v0 = 0.f;
    if (a.gate) {
      // slot s of the pair (CTA r, image b) is r + b; image b owns the slots
      // from its first row's CTA to its last row's
      const int64_t slots = a.rows ? a.ctas + a.images - 1 : 0;
      const double per = (double)a.chunk / ((double)a.chunk + (double)a.tokens);
      for (int64_t s = threadIdx.y; s < slots; s += kColLanes) {
        int64_t b = min((int64_t)(s * per), (int64_t)a.images - 1);
        while (b > 0 && a.tokens * b / a.chunk + b > s) --b;
        while (b + 1 < a.images && a.tokens * (b + 1) / a.chunk + (b + 1) <= s) ++b;
        if ((a.tokens * (b + 1) - 1) / a.chunk + b < s) continue;  // an image ended with its CTA: slot not used
        const float gt = a.gate[b * a.C + cc];
        v1 = fmaf(gt, a.part_post[s * C2 + cc], v1);
        v0 = fmaf(gt, a.part_post[s * C2 + a.C + cc], v0);
      }
    } else {
#pragma unroll 4
      for (int s = threadIdx.y; s < a.ctas; s += kColLanes) {
        v1 += a.part_post[s * C2 + cc];
        v0 += a.part_post[s * C2 + a.C + cc];
      }
    }
    v1 = lane_sum(v1, buf);
    v0 = lane_sum(v0, buf);
    if (own) {
      const float sc = a.scale ? a.scale[c] : 1.f;
      const float gm = a.post_norm && a.gamma ? a.gamma[c] : 1.f, bt = a.post_norm && a.beta ? a.beta[c] : 0.f;
      if (a.dpost_gamma) a.dpost_gamma[c] = sc * v1;
      if (a.dpost_beta) a.dpost_beta[c] = sc * v0;
      if (a.dscale) a.dscale[c] = fmaf(gm, v1, bt * v0);
    }
  }
}

// ---- dropout -------------------------------------------------------------------
// Element i keeps iff decision i / span does. kMode 0: span 1, one block per
// 8-element vector; 1: span a multiple of 8, one decision per vector; 2: any
// other span, one decision per element.
template <typename T, int kMode>
__global__ void __launch_bounds__(256) dropout_kernel(const T *x, T *y, int64_t n, int64_t span, Drop d) {
  Philox ph;
  ph.init(d);
  const int64_t nvec = (n + 7) >> 3;
  for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < nvec; v += (int64_t)gridDim.x * 256) {
    const int64_t i0 = v * 8;
    uint4 bits = make_uint4(0u, 0u, 0u, 0u);
    if (kMode == 0) bits = ph.block((uint64_t)v);
    if (kMode == 1 && keep_one(ph, (uint64_t)(i0 / span), d.thr)) bits = make_uint4(~0u, ~0u, ~0u, ~0u);
    float f[8];
    if (i0 + 8 <= n) {
      unpack(load8<T>(x, v), f);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool keep = kMode == 2 ? keep_one(ph, (uint64_t)((i0 + e) / span), d.thr) : keep_of(bits, e, d.thr);
        f[e] = keep ? f[e] * d.scale : 0.f;
      }
      Raw<T> out;
      pack(f, out);
      store8(y, v, out);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i0 + e < n) {
          const bool keep = kMode == 2 ? keep_one(ph, (uint64_t)((i0 + e) / span), d.thr) : keep_of(bits, e, d.thr);
          y[i0 + e] = (T)(keep ? (float)x[i0 + e] * d.scale : 0.f);
        }
    }
  }
}

// ---- launch shapes ---------------------------------------------------------------
struct Shape {
  int tpr, nv, ctas_per_sm;
};

// Threads per row and vectors per thread: the narrowest that holds the row.
Shape shape_of(int C) {
  const int c8 = C >> 3;
  if (c8 <= 4) return {4, 1, 2};
  if (c8 <= 8) return {8, 1, 2};
  if (c8 <= 16) return {16, 1, 2};
  if (c8 <= 32) return {32, 1, 2};
  if (c8 <= 64) return {32, 2, 1};
  if (c8 <= 128) return {128, 1, 4};
  if (c8 <= 256) return {256, 1, 2};
  if (c8 <= 512) return {256, 2, 1};
  return {512, 2, 1};
}

struct Split {
  int64_t chunk;
  int ctas;
};

Split split_rows(int64_t rows, int C, int sms, int per_sm) {
  const Shape sh = shape_of(C);
  const int64_t at_once = sh.tpr > 32 ? 1 : 256 / sh.tpr;
  const int64_t groups = (rows + at_once - 1) / at_once;
  const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)sms * per_sm));
  int64_t chunk = (rows + ctas - 1) / ctas;
  chunk = std::max<int64_t>(1, (chunk + at_once - 1) / at_once * at_once);
  return {chunk, (int)((rows + chunk - 1) / chunk)};
}

int sm_count(int *sms) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SWIN_ERR_CUDA;
  return SWIN_OK;
}

template <typename T, int TPR, int NV>
int launch_rows(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st) {
  constexpr int t = block_of(TPR);
  if (bwd) {
    if (branch && pre) rows_bwd_kernel<T, TPR, NV, true, true><<<ctas, t, 0, st>>>(a);
    else if (branch) rows_bwd_kernel<T, TPR, NV, true, false><<<ctas, t, 0, st>>>(a);
    else rows_bwd_kernel<T, TPR, NV, false, true><<<ctas, t, 0, st>>>(a);
  } else {
    if (branch && pre) rows_fwd_kernel<T, TPR, NV, true, true><<<ctas, t, 0, st>>>(a);
    else if (branch) rows_fwd_kernel<T, TPR, NV, true, false><<<ctas, t, 0, st>>>(a);
    else rows_fwd_kernel<T, TPR, NV, false, true><<<ctas, t, 0, st>>>(a);
  }
  return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

template <typename T>
int launch_shape(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st) {
  const Shape sh = shape_of(a.C);
  if (sh.tpr == 4) return launch_rows<T, 4, 1>(a, bwd, branch, pre, ctas, st);
  if (sh.tpr == 8) return launch_rows<T, 8, 1>(a, bwd, branch, pre, ctas, st);
  if (sh.tpr == 16) return launch_rows<T, 16, 1>(a, bwd, branch, pre, ctas, st);
  if (sh.tpr == 32 && sh.nv == 1) return launch_rows<T, 32, 1>(a, bwd, branch, pre, ctas, st);
  if (sh.tpr == 32) return launch_rows<T, 32, 2>(a, bwd, branch, pre, ctas, st);
  if (sh.tpr == 128) return launch_rows<T, 128, 1>(a, bwd, branch, pre, ctas, st);
  if (sh.tpr == 256 && sh.nv == 1) return launch_rows<T, 256, 1>(a, bwd, branch, pre, ctas, st);
  if (sh.tpr == 256) return launch_rows<T, 256, 2>(a, bwd, branch, pre, ctas, st);
  return launch_rows<T, 512, 2>(a, bwd, branch, pre, ctas, st);
}

// ---- argument checks ---------------------------------------------------------------
bool mis(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

int check_rows(const swin_attn_rows *r, int64_t *rows, size_t *bytes) {
  if (!r || r->images < 0 || r->tokens < 0) return SWIN_ERR_INVALID_ARG;
  if (r->dtype != SWIN_F32 && r->dtype != SWIN_BF16) return SWIN_ERR_UNSUPPORTED;
  if (r->channels < 8 || r->channels % 8 || r->channels > 8192) return SWIN_ERR_UNSUPPORTED;
  if (r->images > INT32_MAX || r->tokens > INT32_MAX) return SWIN_ERR_UNSUPPORTED;
  *rows = r->images * r->tokens;
  if (*rows > INT32_MAX) return SWIN_ERR_UNSUPPORTED;
  *bytes = (size_t)*rows * r->channels * (r->dtype == SWIN_BF16 ? 2 : 4);
  return SWIN_OK;
}

int check_norm(const swin_attn_norm &n, Norm *out) {
  if (n.kind < SWIN_NORM_NONE || n.kind > SWIN_NORM_RMS) return SWIN_ERR_INVALID_ARG;
  if (n.kind != SWIN_NORM_NONE && (!(n.eps > 0.f) || !std::isfinite(n.eps))) return SWIN_ERR_INVALID_ARG;
  if (mis(n.gamma, 4) || mis(n.beta, 4)) return SWIN_ERR_ALIGNMENT;
  *out = Norm{n.kind, n.eps, n.gamma, n.beta};
  return SWIN_OK;
}

// in may be exactly out; a partial overlap is refused
bool clash(const void *in, const void *out, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(in), b = reinterpret_cast<uintptr_t>(out);
  return in && out && a != b && a < b + bytes && b < a + bytes;
}
bool overlap(const void *p, const void *q, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && a < b + bytes && b < a + bytes;
}

int64_t col_slots(int ctas, int64_t images) { return (int64_t)ctas + std::max<int64_t>(images, 1); }

}  // namespace
}  // namespace swin

using namespace swin;

extern "C" {

size_t swin_attn_rows_workspace_bytes(const swin_attn_rows *r) {
  int64_t rows = 0;
  size_t bytes = 0;
  int sms = 0;
  if (check_rows(r, &rows, &bytes) || sm_count(&sms)) return 0;
  const Split sp = split_rows(rows, r->channels, sms, shape_of(r->channels).ctas_per_sm);
  const size_t need = ((size_t)sp.ctas + (size_t)col_slots(sp.ctas, r->images)) * 2 * r->channels * sizeof(float);
  return (need + 255) & ~size_t(255);
}

int swin_attn_norm_fwd(const swin_attn_rows *r, const void *x, const swin_attn_norm *norm, void *h,
                       swin_stream_t stream) {
  RowArgs a = {};
  size_t bytes = 0;
  int rc = check_rows(r, &a.rows, &bytes);
  if (rc) return rc;
  if (!norm || norm->kind == SWIN_NORM_NONE) return SWIN_ERR_INVALID_ARG;
  rc = check_norm(*norm, &a.pre);
  if (rc) return rc;
  if (a.rows == 0) return SWIN_OK;
  if (!x || !h || clash(x, h, bytes)) return SWIN_ERR_INVALID_ARG;
  if (mis(x, 16) || mis(h, 16)) return SWIN_ERR_ALIGNMENT;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc) return rc;
  a.x = x;
  a.h = h;
  a.tokens = a.rows;
  a.images = 1;
  a.C = r->channels;
  a.path.scale = a.drop.scale = 1.f;
  const Split sp = split_rows(a.rows, a.C, sms, 4 * shape_of(a.C).ctas_per_sm);
  a.chunk = sp.chunk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return r->dtype == SWIN_BF16 ? launch_shape<__nv_bfloat16>(a, false, false, true, sp.ctas, st)
                               : launch_shape<float>(a, false, false, true, sp.ctas, st);
}

int swin_attn_join_fwd(const swin_attn_rows *r, const void *x, const void *z, const swin_attn_join *join, void *y,
                       void *h, swin_stream_t stream) {
  RowArgs a = {};
  size_t bytes = 0;
  int rc = check_rows(r, &a.rows, &bytes);
  if (rc) return rc;
  if (!join) return SWIN_ERR_INVALID_ARG;
  if ((rc = check_norm(join->post, &a.post)) || (rc = check_norm(join->pre, &a.pre)) ||
      (rc = make_drop(&join->drop, &a.drop)) || (rc = make_drop(&join->path, &a.path)))
    return rc;
  const bool pre = a.pre.kind != SWIN_NORM_NONE;
  if (!pre && h) return SWIN_ERR_INVALID_ARG;
  if (mis(join->scale, 4) || mis(join->gate, 4)) return SWIN_ERR_ALIGNMENT;
  if (a.rows == 0) return SWIN_OK;
  if (!x || !z || !y || (pre && !h)) return SWIN_ERR_INVALID_ARG;
  if (clash(x, y, bytes) || clash(z, y, bytes) || clash(x, h, bytes) || clash(z, h, bytes) || overlap(y, h, bytes))
    return SWIN_ERR_INVALID_ARG;
  if (mis(x, 16) || mis(z, 16) || mis(y, 16) || mis(h, 16)) return SWIN_ERR_ALIGNMENT;
  int sms = 0;
  rc = sm_count(&sms);
  if (rc) return rc;
  a.x = x;
  a.z = z;
  a.y = y;
  a.h = h;
  a.scale = join->scale;
  a.gate = join->gate;
  a.tokens = r->tokens;
  a.images = (int)r->images;
  a.C = r->channels;
  const Split sp = split_rows(a.rows, a.C, sms, 4 * shape_of(a.C).ctas_per_sm);
  a.chunk = sp.chunk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return r->dtype == SWIN_BF16 ? launch_shape<__nv_bfloat16>(a, false, true, pre, sp.ctas, st)
                               : launch_shape<float>(a, false, true, pre, sp.ctas, st);
}

}  // extern "C"

namespace {

// Row pass and parameter gradients of the two backward entry points.
int run_backward(RowArgs &a, const swin_attn_rows *r, bool branch, const swin_attn_join_grads &g, void *workspace,
                 size_t workspace_bytes, cudaStream_t st) {
  const bool pre = a.pre.kind != SWIN_NORM_NONE, post = a.post.kind != SWIN_NORM_NONE;
  const bool want_pre = pre && (g.pre_gamma || g.pre_beta);
  const bool want_post = branch && (g.post_gamma || g.post_beta || g.scale || g.gate);
  int sms = 0;
  int rc = sm_count(&sms);
  if (rc) return rc;
  a.C = r->channels;
  a.images = (int)r->images;
  a.tokens = branch ? r->tokens : a.rows;  // the norm alone does not look at images
  const Split sp = split_rows(a.rows, a.C, sms, shape_of(a.C).ctas_per_sm);
  a.chunk = sp.chunk;
  if (want_pre || want_post) {
    if (!workspace || workspace_bytes < swin_attn_rows_workspace_bytes(r)) return SWIN_ERR_WORKSPACE;
    if (mis(workspace, 256)) return SWIN_ERR_ALIGNMENT;
    float *ws = static_cast<float *>(workspace);
    a.part_pre = want_pre ? ws : nullptr;
    a.part_post = want_post ? ws + (size_t)sp.ctas * 2 * a.C : nullptr;
  }
  if (a.rows) {
    rc = r->dtype == SWIN_BF16 ? launch_shape<__nv_bfloat16>(a, true, branch, pre, sp.ctas, st)
                               : launch_shape<float>(a, true, branch, pre, sp.ctas, st);
    if (rc) return rc;
  }
  if (!want_pre && !want_post) return SWIN_OK;
  ColArgs c = {};
  c.rows = a.rows;
  c.tokens = a.tokens;
  c.chunk = a.chunk;
  c.images = a.images;
  c.C = a.C;
  c.ctas = a.rows ? sp.ctas : 0;
  c.post_norm = post;
  c.part_pre = a.part_pre;
  c.part_post = a.part_post;
  c.scale = a.scale;
  c.gate = a.gate;
  c.gamma = a.post.gamma;
  c.beta = a.post.beta;
  if (want_pre) {
    c.dpre_gamma = g.pre_gamma;
    c.dpre_beta = g.pre_beta;
  }
  if (want_post) {
    c.dpost_gamma = post ? g.post_gamma : nullptr;
    c.dpost_beta = post ? g.post_beta : nullptr;
    c.dscale = g.scale;
    c.dgate = g.gate;
  }
  const int64_t tiles = (a.C + 31) / 32;
  const int64_t blocks = tiles * (1 + (c.dgate ? (int64_t)a.images : 0));
  if (blocks > INT32_MAX) return SWIN_ERR_UNSUPPORTED;
  columns_kernel<<<(int)blocks, dim3(32, kColLanes), 0, st>>>(c);
  return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

}  // namespace

extern "C" {

int swin_attn_norm_bwd(const swin_attn_rows *r, const void *x, const swin_attn_norm *norm, const void *dh,
                       const void *dres, void *dx, float *dgamma, float *dbeta, void *workspace,
                       size_t workspace_bytes, swin_stream_t stream) {
  RowArgs a = {};
  size_t bytes = 0;
  int rc = check_rows(r, &a.rows, &bytes);
  if (rc) return rc;
  if (!norm || norm->kind == SWIN_NORM_NONE) return SWIN_ERR_INVALID_ARG;
  rc = check_norm(*norm, &a.pre);
  if (rc) return rc;
  if (mis(dgamma, 4) || mis(dbeta, 4)) return SWIN_ERR_ALIGNMENT;
  if (a.rows) {
    if (!x || !dh || !dx) return SWIN_ERR_INVALID_ARG;
    if (clash(x, dx, bytes) || clash(dh, dx, bytes) || clash(dres, dx, bytes)) return SWIN_ERR_INVALID_ARG;
    if (mis(x, 16) || mis(dh, 16) || mis(dres, 16) || mis(dx, 16)) return SWIN_ERR_ALIGNMENT;
  }
  a.x = x;
  a.dh = dh;
  a.dy = dres;
  a.dx = dx;
  a.path.scale = a.drop.scale = 1.f;
  swin_attn_join_grads g = {};
  g.pre_gamma = dgamma;
  g.pre_beta = dbeta;
  return run_backward(a, r, false, g, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

int swin_attn_join_bwd(const swin_attn_rows *r, const void *y, const void *z, const swin_attn_join *join,
                       const void *dy, const void *dh, void *dx, void *dz, const swin_attn_join_grads *grads,
                       void *workspace, size_t workspace_bytes, swin_stream_t stream) {
  RowArgs a = {};
  size_t bytes = 0;
  int rc = check_rows(r, &a.rows, &bytes);
  if (rc) return rc;
  if (!join || !grads) return SWIN_ERR_INVALID_ARG;
  if ((rc = check_norm(join->post, &a.post)) || (rc = check_norm(join->pre, &a.pre)) ||
      (rc = make_drop(&join->drop, &a.drop)) || (rc = make_drop(&join->path, &a.path)))
    return rc;
  const bool pre = a.pre.kind != SWIN_NORM_NONE, post = a.post.kind != SWIN_NORM_NONE;
  if ((!pre && (dh || grads->pre_gamma || grads->pre_beta)) || (!post && (grads->post_gamma || grads->post_beta)) ||
      (grads->gate && !join->gate))
    return SWIN_ERR_INVALID_ARG;
  const float *small[8] = {join->scale,      join->gate,  grads->post_gamma, grads->post_beta,
                           grads->scale, grads->gate, grads->pre_gamma,  grads->pre_beta};
  for (const float *p : small)
    if (mis(p, 4)) return SWIN_ERR_ALIGNMENT;
  const bool need_z = post || grads->scale || grads->gate;
  if (a.rows) {
    if ((!dy && !dh) || !dx || !dz || (need_z && !z) || (dh && !y)) return SWIN_ERR_INVALID_ARG;
    const void *in[4] = {y, z, dy, dh};
    for (const void *p : in) {
      if (clash(p, dx, bytes) || clash(p, dz, bytes)) return SWIN_ERR_INVALID_ARG;
      if (mis(p, 16)) return SWIN_ERR_ALIGNMENT;
    }
    if (overlap(dx, dz, bytes)) return SWIN_ERR_INVALID_ARG;
    if (mis(dx, 16) || mis(dz, 16)) return SWIN_ERR_ALIGNMENT;
  }
  if (!dh) a.pre.kind = SWIN_NORM_NONE;  // nothing reached h: its norm's gradients are zero
  a.x = y;
  a.z = need_z ? z : nullptr;
  a.dy = dy;
  a.dh = dh;
  a.dx = dx;
  a.dz = dz;
  a.scale = join->scale;
  a.gate = join->gate;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (pre && !dh) {
    const size_t cb = sizeof(float) * r->channels;
    if (grads->pre_gamma && cudaMemsetAsync(grads->pre_gamma, 0, cb, st) != cudaSuccess) return SWIN_ERR_CUDA;
    if (grads->pre_beta && cudaMemsetAsync(grads->pre_beta, 0, cb, st) != cudaSuccess) return SWIN_ERR_CUDA;
  }
  return run_backward(a, r, true, *grads, workspace, workspace_bytes, st);
}

int swin_attn_dropout(int32_t dtype, int64_t n, int64_t span, const void *x, const swin_attn_drop *drop, void *y,
                      swin_stream_t stream) {
  if (n < 0 || span < 1 || n > (int64_t(1) << 46)) return SWIN_ERR_INVALID_ARG;
  if (dtype != SWIN_F32 && dtype != SWIN_BF16) return SWIN_ERR_UNSUPPORTED;
  Drop d;
  int rc = make_drop(drop, &d);
  if (rc) return rc;
  if (n == 0) return SWIN_OK;
  const size_t bytes = (size_t)n * (dtype == SWIN_BF16 ? 2 : 4);
  if (!x || !y || clash(x, y, bytes)) return SWIN_ERR_INVALID_ARG;
  if (mis(x, 16) || mis(y, 16)) return SWIN_ERR_ALIGNMENT;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!d.thr) {  // rate 0
    if (x != y && cudaMemcpyAsync(y, x, bytes, cudaMemcpyDeviceToDevice, st) != cudaSuccess) return SWIN_ERR_CUDA;
    return SWIN_OK;
  }
  int sms = 0;
  rc = sm_count(&sms);
  if (rc) return rc;
  const int64_t nvec = (n + 7) / 8;
  const int blocks = (int)std::min<int64_t>((nvec + 255) / 256, (int64_t)sms * 8);
  const int mode = span == 1 ? 0 : span % 8 == 0 ? 1 : 2;
  if (dtype == SWIN_BF16) {
    const __nv_bfloat16 *p = static_cast<const __nv_bfloat16 *>(x);
    __nv_bfloat16 *q = static_cast<__nv_bfloat16 *>(y);
    if (mode == 0) dropout_kernel<__nv_bfloat16, 0><<<blocks, 256, 0, st>>>(p, q, n, span, d);
    else if (mode == 1) dropout_kernel<__nv_bfloat16, 1><<<blocks, 256, 0, st>>>(p, q, n, span, d);
    else dropout_kernel<__nv_bfloat16, 2><<<blocks, 256, 0, st>>>(p, q, n, span, d);
  } else {
    const float *p = static_cast<const float *>(x);
    float *q = static_cast<float *>(y);
    if (mode == 0) dropout_kernel<float, 0><<<blocks, 256, 0, st>>>(p, q, n, span, d);
    else if (mode == 1) dropout_kernel<float, 1><<<blocks, 256, 0, st>>>(p, q, n, span, d);
    else dropout_kernel<float, 2><<<blocks, 256, 0, st>>>(p, q, n, span, d);
  }
  return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

}  // extern "C"
