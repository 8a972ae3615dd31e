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
// A vector is 8 channels: 16 bytes of bf16, 32 of fp32. In registers it is four
// float2, the operands of the packed fp32 instructions (two results an issue).
template <typename T>
constexpr int vec_bytes() { return 8 * (int)sizeof(T); }

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

__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16> &r, float2 (&f)[4]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const Raw<float> &r, float2 (&f)[4]) {
  f[0] = make_float2(r.a.x, r.a.y), f[1] = make_float2(r.a.z, r.a.w);
  f[2] = make_float2(r.b.x, r.b.y), f[3] = make_float2(r.b.z, r.b.w);
}

__device__ __forceinline__ void pack(const float2 (&f)[4], Raw<__nv_bfloat16> &r) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[e].x, f[e].y);
    w[e] = *reinterpret_cast<const uint32_t *>(&h);
  }
  r.v = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack(const float2 (&f)[4], Raw<float> &r) {
  r.a = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  r.b = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
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
__device__ __forceinline__ void load_param(const float *p, int vec, bool ok, float none, float2 (&f)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    f[e] = p && ok ? make_float2(__ldg(p + 8 * vec + 2 * e), __ldg(p + 8 * vec + 2 * e + 1)) : make_float2(none, none);
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
// Pair e (0..3) of a vector where the decisions of its generator block keep, else 0.
__device__ __forceinline__ float2 kept(const uint4 &bits, int e, uint32_t thr, float2 v) {
  return make_float2(keep_of(bits, 2 * e, thr) ? v.x : 0.f, keep_of(bits, 2 * e + 1, thr) ? v.y : 0.f);
}

// ---- the ring ------------------------------------------------------------------
// Rows come through a ring of D + 1 stages in shared memory, D rows ahead, by
// 16-byte asynchronous copies (cp.async). Every thread copies exactly the
// vectors that it reads back, so the ring needs no barrier, only the thread's
// own wait for its copies; the bytes in flight no longer depend on how many
// registers a warp's work takes.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Slot (stage, tensor, vector j) of this thread: 16-byte pieces of consecutive
// threads are consecutive (no bank conflicts).
template <typename T, int kThreads, int NT, int NV>
struct Ring {
  static constexpr int kPieces = vec_bytes<T>() / 16;
  static constexpr int kStage = kThreads * NT * NV * vec_bytes<T>();
  uint8_t *base;
  uint32_t addr;
  __device__ __forceinline__ void init(uint8_t *smem) {
    base = smem + threadIdx.x * 16;
    addr = static_cast<uint32_t>(__cvta_generic_to_shared(base));
  }
  static __device__ __forceinline__ int slot(int stage, int t, int j) {
    return stage * kStage + (t * NV + j) * kPieces * kThreads * 16;
  }
  // a vector of a tensor (its first byte's place if it is not there: nothing is read, zeros arrive)
  __device__ __forceinline__ void fetch(int stage, int t, int j, const void *tensor, int64_t vec, bool there) const {
    const uint8_t *src = static_cast<const uint8_t *>(tensor) + (there ? vec * vec_bytes<T>() : 0);
#pragma unroll
    for (int p = 0; p < kPieces; ++p) copy16(addr + slot(stage, t, j) + p * kThreads * 16, src + 16 * p, there);
  }
  __device__ __forceinline__ void read(int stage, int t, int j, float2 (&f)[4]) const {
    const uint8_t *p = base + slot(stage, t, j);
    Raw<T> r;
    if constexpr (kPieces == 1) {
      r.v = *reinterpret_cast<const uint4 *>(p);
    } else {
      r.a = *reinterpret_cast<const float4 *>(p);
      r.b = *reinterpret_cast<const float4 *>(p + kThreads * 16);
    }
    unpack(r, f);
  }
};

// ---- launch shapes ----------------------------------------------------------------
// One kernel's shape: TPR threads a row with NV vectors each, NT input tensors.
constexpr int block_of(int tpr) { return tpr > 32 ? tpr : 256; }

// Resident CTAs an SM (and the register bound that allows them). Backward: four
// column sums, two parameters and four rows of 8 channels are 80 registers
// before any address, so 512 threads with 128 registers; twice that for two
// vectors.
constexpr int blocks_per_sm(int tpr, int nv, bool bwd) {
  return bwd ? (nv == 2 ? 1 : 512 / block_of(tpr)) : (nv == 2 ? 512 : 768) / block_of(tpr);
}

// Rows ahead: 64 KB in flight on an SM cover HBM's latency at its rate (about
// 1 us at 45 GB/s a SM), as far as 200 KB of shared memory hold the ring.
constexpr int rows_ahead(int stage_bytes, int blocks) {
  int d = (65536 + blocks * stage_bytes - 1) / (blocks * stage_bytes);
  const int most = 200 * 1024 / blocks / stage_bytes - 1;
  d = d > most ? most : d;
  return d < 0 ? 0 : d > 7 ? 7 : d;
}

template <typename T, int TPR, int NV, bool kBwd, bool kBranch, bool kPre>
struct Shape {
  static constexpr int threads = block_of(TPR);
  static constexpr int blocks = blocks_per_sm(TPR, NV, kBwd);
  static constexpr int tensors = kBwd ? 1 + (kPre ? 2 : 0) + (kBranch ? 1 : 0) : (kBranch ? 2 : 1);
  static constexpr int stage = threads * tensors * NV * vec_bytes<T>();
  static constexpr int ahead = rows_ahead(stage, blocks);
  static constexpr int flush = kBwd && TPR <= 32 ? threads * NV * 32 : 0;
  static constexpr int smem = (ahead + 1) * stage > flush ? (ahead + 1) * stage : flush;
  static_assert(smem <= 227 * 1024, "over a CTA's shared memory");
};

// ---- sums over a row ---------------------------------------------------------
// Sums of a pair over the TPR threads of a row. Rows of up to 32 threads stay
// inside a warp; wider rows are the whole CTA and exchange one pair per warp
// through one of two shared buffers (used in turn: one barrier per sum).
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 v, float2 *xchg, int &turn) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1)
    v = add(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    float2 *buf = xchg + turn * W;
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = add(v, buf[w]);
  }
  return v;
}

template <int NV>
__device__ __forceinline__ float sum_of(const float2 (&u)[NV][4]) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = add(s, u[j][e]);
  return s.x + s.y;
}
template <int NV>
__device__ __forceinline__ float dot_of(const float2 (&u)[NV][4], const float2 (&v)[NV][4]) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) s = fma(u[j][e], v[j][e], s);
  return s.x + s.y;
}
// u - m; vectors past the row's end stay 0
template <int NV>
__device__ __forceinline__ void centre(float2 (&u)[NV][4], float m, const bool (&ok)[NV]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const float2 n = both(ok[j] ? -m : 0.f);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[j][e] = add(u[j][e], n);
  }
}

// Where a CTA's rows lie and which of them a thread works on.
struct Place {
  int lane, sub;
  int64_t first, stride;
};
template <int TPR>
__device__ __forceinline__ Place place() {
  constexpr int kWarps = block_of(TPR) / 32, RPW = TPR < 32 ? 32 / TPR : 1;  // rows a warp works on at once
  Place p;
  p.lane = TPR > 32 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  p.sub = TPR < 32 ? (threadIdx.x & 31) / TPR : 0;
  p.first = TPR > 32 ? 0 : (threadIdx.x >> 5) * RPW;
  p.stride = TPR > 32 ? 1 : kWarps * RPW;
  return p;
}

// ---- forward -----------------------------------------------------------------
template <typename T, int TPR, int NV, bool kBranch, bool kPre>
__global__ void __launch_bounds__(block_of(TPR), blocks_per_sm(TPR, NV, false)) rows_fwd_kernel(const RowArgs a) {
  using S = Shape<T, TPR, NV, false, kBranch, kPre>;
  constexpr int D = S::ahead;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 xchg[TPR > 32 ? 2 * (TPR / 32) : 1];
  int turn = 0;
  const Place pl = place<TPR>();
  const int C8 = a.C >> 3;
  const float inv = 1.0f / (float)a.C;
  Ring<T, S::threads, S::tensors, NV> ring;
  ring.init(smem);
  bool ok[NV];
  float2 gpre[NV][4], bpre[NV][4], wg[NV][4], wb[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    ok[j] = j * TPR + pl.lane < C8;
    if constexpr (kPre) {
      load_param(a.pre.gamma, j * TPR + pl.lane, ok[j], 1.f, gpre[j]);
      load_param(a.pre.beta, j * TPR + pl.lane, ok[j], 0.f, bpre[j]);
    }
  }
  Philox ph;
  ph.init(a.drop);
  const bool post = a.post.kind != SWIN_NORM_NONE;

  const int64_t L = (int64_t)blockIdx.x * a.chunk;
  const int64_t R = min(L + a.chunk, a.rows);
  // one image of the CTA's rows at a time: the gate and the path decision change with it
  for (int64_t s = L; s < R;) {
    const int64_t b = s / a.tokens;
    const int64_t e1 = min(R, (b + 1) * a.tokens);
    auto fetch = [&](int64_t r0, int stage) {
      const int64_t row = r0 + pl.sub, vec0 = row * C8 + pl.lane;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const bool there = ok[j] && row < e1;
        ring.fetch(stage, 0, j, a.x, vec0 + j * TPR, there);
        if constexpr (kBranch) ring.fetch(stage, 1, j, a.z, vec0 + j * TPR, there);
      }
      copies_commit();
    };
    int64_t ahead = s + pl.first;
    int in = 0, out = 0;
#pragma unroll
    for (int k = 0; k < D; ++k, ahead += pl.stride) fetch(ahead, in++);
    bool path = true;
    if constexpr (kBranch) {
      float c = a.drop.scale;  // what is kept is multiplied by, with the gate and the layer scale
      if (a.path.thr) {
        Philox pp;
        pp.init(a.path);
        path = keep_one(pp, (uint64_t)b, a.path.thr);
        c *= a.path.scale;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float2 t[4];
        load_param(a.scale, j * TPR + pl.lane, ok[j], 1.f, wg[j]);
        load_param(a.gate ? a.gate + b * a.C : nullptr, j * TPR + pl.lane, ok[j], 1.f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) wb[j][e] = wg[j][e] = mul(mul(wg[j][e], t[e]), both(c));
        load_param(a.post.gamma, j * TPR + pl.lane, ok[j] && post, 1.f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) wg[j][e] = mul(wg[j][e], t[e]);
        load_param(a.post.beta, j * TPR + pl.lane, ok[j] && post, 0.f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) wb[j][e] = mul(wb[j][e], t[e]);
      }
    }
    for (int64_t r0 = s + pl.first; r0 < e1; r0 += pl.stride, ahead += pl.stride) {
      fetch(ahead, in);
      in = in == D ? 0 : in + 1;
      copies_wait<D>();
      const int64_t row = r0 + pl.sub;
      const bool live = row < e1;
      const int64_t vec0 = row * C8 + pl.lane;
      float2 v[NV][4];
#pragma unroll
      for (int j = 0; j < NV; ++j) ring.read(out, 0, j, v[j]);
      if constexpr (kBranch) {
        float2 u[NV][4];
#pragma unroll
        for (int j = 0; j < NV; ++j) ring.read(out, 1, j, u[j]);
        float2 rstd = both(1.f);
        if (post) {
          if (a.post.kind == SWIN_NORM_LAYER)
            centre<NV>(u, row_sum<TPR>(make_float2(sum_of<NV>(u), 0.f), xchg, turn).x * inv, ok);
          rstd = both(rsqrtf(fmaf(row_sum<TPR>(make_float2(dot_of<NV>(u, u), 0.f), xchg, turn).x, inv, a.post.eps)));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (path) {  // a dropped image's y is x
            uint4 bits;
            if (a.drop.thr) bits = ph.block((uint64_t)(vec0 + j * TPR));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float2 br = fma(mul(u[j][e], rstd), wg[j][e], wb[j][e]);
              if (a.drop.thr) br = kept(bits, e, a.drop.thr, br);
              v[j][e] = add(v[j][e], br);
            }
          }
          Raw<T> o;
          pack(v[j], o);
          if (ok[j] && live) store8(a.y, vec0 + j * TPR, o);
          if constexpr (kPre) unpack(o, v[j]);  // h is the norm of y as stored
        }
      }
      out = out == D ? 0 : out + 1;
      if constexpr (kPre) {
        if (a.pre.kind == SWIN_NORM_LAYER)
          centre<NV>(v, row_sum<TPR>(make_float2(sum_of<NV>(v), 0.f), xchg, turn).x * inv, ok);
        const float2 rstd =
            both(rsqrtf(fmaf(row_sum<TPR>(make_float2(dot_of<NV>(v, v), 0.f), xchg, turn).x, inv, a.pre.eps)));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          Raw<T> o;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] = fma(mul(v[j][e], rstd), gpre[j][e], bpre[j][e]);
          pack(v[j], o);
          if (ok[j] && live) store8(a.h, vec0 + j * TPR, o);
        }
      }
    }
    copies_wait<0>();
    s = e1;
  }
}

// ---- backward ----------------------------------------------------------------
// Sums the CTA's copies of this thread's channels and writes them: dst[C].
template <int TPR, int NV>
__device__ __forceinline__ void flush(float2 (&acc)[NV][4], float *dst, int C8, float *buf) {
  constexpr int kThreads = block_of(TPR);
  const int lane = TPR > 32 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  auto put = [&](float *p, const float2 (&v)[4]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  };
  if constexpr (TPR > 32) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j * TPR + lane < C8) put(dst + 8 * (j * TPR + lane), acc[j]);
  } else {
    constexpr int G = kThreads / TPR, W = TPR * NV * 8;  // rows in flight, channels of a row (padded)
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) put(buf + threadIdx.x / TPR * W + 8 * (j * TPR + lane), acc[j]);
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
    for (int e = 0; e < 4; ++e) acc[j][e] = make_float2(0.f, 0.f);
}

template <typename T, int TPR, int NV, bool kBranch, bool kPre>
__global__ void __launch_bounds__(block_of(TPR), blocks_per_sm(TPR, NV, true)) rows_bwd_kernel(const RowArgs a) {
  using S = Shape<T, TPR, NV, true, kBranch, kPre>;
  constexpr int D = S::ahead;
  constexpr int tDy = 0, tY = 1, tDh = 2, tZ = kPre ? 3 : 1;  // tensors of a stage
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 xchg[TPR > 32 ? 2 * (TPR / 32) : 1];
  int turn = 0;
  const Place pl = place<TPR>();
  const int C8 = a.C >> 3;
  const float inv = 1.0f / (float)a.C;
  Ring<T, S::threads, S::tensors, NV> ring;
  ring.init(smem);
  bool ok[NV];
  float2 gpre[NV][4], w[NV][4];
  float2 a1[NV][4], a0[NV][4], b1[NV][4], b0[NV][4];  // column sums: dh yhat, dh; G zhat, G
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    ok[j] = j * TPR + pl.lane < C8;
    if constexpr (kPre) load_param(a.pre.gamma, j * TPR + pl.lane, ok[j], 1.f, gpre[j]);
#pragma unroll
    for (int e = 0; e < 4; ++e) a1[j][e] = a0[j][e] = b1[j][e] = b0[j][e] = make_float2(0.f, 0.f);
  }
  Philox ph;
  ph.init(a.drop);
  const bool post = a.post.kind != SWIN_NORM_NONE;

  const int64_t L = (int64_t)blockIdx.x * a.chunk;
  const int64_t R = min(L + a.chunk, a.rows);
  for (int64_t s = L; s < R;) {
    const int64_t b = s / a.tokens;
    const int64_t e1 = min(R, (b + 1) * a.tokens);
    auto fetch = [&](int64_t r0, int stage) {
      const int64_t row = r0 + pl.sub, vec0 = row * C8 + pl.lane;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const bool there = ok[j] && row < e1;
        if (a.dy) ring.fetch(stage, tDy, j, a.dy, vec0 + j * TPR, there);
        if constexpr (kPre) {
          ring.fetch(stage, tY, j, a.x, vec0 + j * TPR, there);
          ring.fetch(stage, tDh, j, a.dh, vec0 + j * TPR, there);
        }
        if constexpr (kBranch)
          if (a.z) ring.fetch(stage, tZ, j, a.z, vec0 + j * TPR, there);
      }
      copies_commit();
    };
    int64_t ahead = s + pl.first;
    int in = 0, out = 0;
#pragma unroll
    for (int k = 0; k < D; ++k, ahead += pl.stride) fetch(ahead, in++);
    bool path = true;
    if constexpr (kBranch) {
      float c = a.drop.scale;  // the kept values' scales: in dz here, in the column sums at the fold
      if (a.path.thr) {
        Philox pp;
        pp.init(a.path);
        path = keep_one(pp, (uint64_t)b, a.path.thr);
        c *= a.path.scale;
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float2 t[4];
        load_param(a.scale, j * TPR + pl.lane, ok[j], 1.f, w[j]);
        load_param(a.gate ? a.gate + b * a.C : nullptr, j * TPR + pl.lane, ok[j], 1.f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[j][e] = mul(mul(w[j][e], t[e]), both(c));
        load_param(a.post.gamma, j * TPR + pl.lane, ok[j] && post, 1.f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[j][e] = mul(w[j][e], t[e]);
      }
    }
    for (int64_t r0 = s + pl.first; r0 < e1; r0 += pl.stride, ahead += pl.stride) {
      fetch(ahead, in);
      in = in == D ? 0 : in + 1;
      copies_wait<D>();
      const int64_t row = r0 + pl.sub;
      const bool live = row < e1;  // rows past the end arrived as zeros and add nothing to the sums
      const int64_t vec0 = row * C8 + pl.lane;
      float2 g[NV][4];  // dy, then dy' = dx
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (a.dy) {
          ring.read(out, tDy, j, g[j]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) g[j][e] = make_float2(0.f, 0.f);
        }
      }
      if constexpr (kPre) {
        float2 u[NV][4], dh[NV][4];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          ring.read(out, tY, j, u[j]);
          ring.read(out, tDh, j, dh[j]);
        }
        const bool layer = a.pre.kind == SWIN_NORM_LAYER;
        if (layer) centre<NV>(u, row_sum<TPR>(make_float2(sum_of<NV>(u), 0.f), xchg, turn).x * inv, ok);
        const float rstd = rsqrtf(fmaf(row_sum<TPR>(make_float2(dot_of<NV>(u, u), 0.f), xchg, turn).x, inv, a.pre.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            u[j][e] = mul(u[j][e], both(rstd));
            a1[j][e] = fma(dh[j][e], u[j][e], a1[j][e]);
            a0[j][e] = add(a0[j][e], dh[j][e]);
            dh[j][e] = mul(dh[j][e], gpre[j][e]);
          }
        const float2 c = row_sum<TPR>(make_float2(dot_of<NV>(dh, u), layer ? sum_of<NV>(dh) : 0.f), xchg, turn);
        const float2 c1 = both(-c.x * inv), c0 = both(-c.y * inv);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            g[j][e] = fma(both(rstd), add(dh[j][e], fma(u[j][e], c1, c0)), g[j][e]);
      }
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Raw<T> o;
        pack(g[j], o);
        if (ok[j] && live) store8(a.dx, vec0 + j * TPR, o);
      }
      if constexpr (kBranch) {
        float2 u[NV][4];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (a.z && path) {
            ring.read(out, tZ, j, u[j]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) u[j][e] = make_float2(0.f, 0.f);
          }
        }
        const bool layer = a.post.kind == SWIN_NORM_LAYER;
        float rstd = 1.f;
        if (layer) centre<NV>(u, row_sum<TPR>(make_float2(sum_of<NV>(u), 0.f), xchg, turn).x * inv, ok);
        if (post) rstd = rsqrtf(fmaf(row_sum<TPR>(make_float2(dot_of<NV>(u, u), 0.f), xchg, turn).x, inv, a.post.eps));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const bool in_row = ok[j] && live;  // past the row's end dy' is not 0
          uint4 bits;
          if (a.drop.thr) bits = ph.block((uint64_t)(vec0 + j * TPR));
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            u[j][e] = mul(u[j][e], both(rstd));
            if (!path || !in_row) g[j][e] = make_float2(0.f, 0.f);
            if (a.drop.thr) {
              g[j][e] = kept(bits, e, a.drop.thr, g[j][e]);
              // what was dropped takes no part, were it infinite (a row's norm has it in its statistics anyway)
              if (!post) u[j][e] = kept(bits, e, a.drop.thr, u[j][e]);
            }
            b1[j][e] = fma(g[j][e], u[j][e], b1[j][e]);
            b0[j][e] = add(b0[j][e], g[j][e]);
            g[j][e] = mul(g[j][e], w[j][e]);
          }
        }
        if (post) {
          const float2 c = row_sum<TPR>(make_float2(dot_of<NV>(g, u), layer ? sum_of<NV>(g) : 0.f), xchg, turn);
          const float2 c1 = both(-c.x * inv), c0 = both(-c.y * inv);
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) g[j][e] = mul(both(rstd), add(g[j][e], fma(u[j][e], c1, c0)));
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          Raw<T> o;
          pack(g[j], o);
          if (ok[j] && live) store8(a.dz, vec0 + j * TPR, o);
        }
      }
      out = out == D ? 0 : out + 1;
    }
    copies_wait<0>();
    // with a gate the sums are kept per image: slot CTA + image (a CTA's next
    // image takes its next slot, the next CTA's first is one further)
    if constexpr (kBranch)
      if (a.part_post && (a.gate || e1 == R)) {
        float *dst = a.part_post + ((int64_t)blockIdx.x + (a.gate ? b : 0)) * 2 * a.C;
        flush<TPR, NV>(b1, dst, C8, reinterpret_cast<float *>(smem));
        flush<TPR, NV>(b0, dst + a.C, C8, reinterpret_cast<float *>(smem));
        if (TPR <= 32) __syncthreads();  // the ring takes the buffer again
      }
    s = e1;
  }
  if constexpr (kPre)
    if (a.part_pre) {
      float *dst = a.part_pre + (int64_t)blockIdx.x * 2 * a.C;
      flush<TPR, NV>(a1, dst, C8, reinterpret_cast<float *>(smem));
      flush<TPR, NV>(a0, dst + a.C, C8, reinterpret_cast<float *>(smem));
    }
}

// ---- parameter gradients from the column sums ----------------------------------
struct ColArgs {
  int64_t tokens, chunk, rows;
  int images, C, ctas;
  bool post_norm;
  float kept;  // what kept values are multiplied by (left out of the join's sums)
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
    v1 = a.kept * lane_sum(v1, buf);
    v0 = a.kept * lane_sum(v0, buf);
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
    v1 = a.kept * lane_sum(v1, buf);
    v0 = a.kept * lane_sum(v0, buf);
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
    if (i0 + 8 <= n) {
      const Raw<T> in = *reinterpret_cast<const Raw<T> *>(x + i0);
      float2 f[4];
      unpack(in, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = mul(f[e], both(d.scale));
        if (kMode == 2) {
          f[e].x = keep_one(ph, (uint64_t)((i0 + 2 * e) / span), d.thr) ? f[e].x : 0.f;
          f[e].y = keep_one(ph, (uint64_t)((i0 + 2 * e + 1) / span), d.thr) ? f[e].y : 0.f;
        } else {
          f[e] = kept(bits, e, d.thr, f[e]);
        }
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

// ---- launches ----------------------------------------------------------------------
struct Width {
  int tpr, nv;
};

// Threads per row and vectors per thread: the narrowest that holds the row.
Width width_of(int C) {
  const int c8 = C >> 3;
  if (c8 <= 4) return {4, 1};
  if (c8 <= 8) return {8, 1};
  if (c8 <= 16) return {16, 1};
  if (c8 <= 32) return {32, 1};
  if (c8 <= 64) return {32, 2};
  if (c8 <= 128) return {128, 1};
  if (c8 <= 256) return {256, 1};
  if (c8 <= 512) return {256, 2};
  return {512, 2};
}

struct Split {
  int64_t chunk;
  int ctas;
};

// Consecutive rows per CTA, as many CTAs as fit on the GPU at once.
Split split_rows(int64_t rows, int C, int sms, bool bwd) {
  const Width wd = width_of(C);
  const int64_t at_once = wd.tpr > 32 ? 1 : 256 / wd.tpr;
  const int64_t groups = (rows + at_once - 1) / at_once;
  const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)sms * blocks_per_sm(wd.tpr, wd.nv, bwd)));
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

template <typename T, int TPR, int NV, bool kBwd, bool kBranch, bool kPre>
int launch_one(const RowArgs &a, int ctas, cudaStream_t st) {
  using S = Shape<T, TPR, NV, kBwd, kBranch, kPre>;
  void (*kern)(const RowArgs);
  if constexpr (kBwd) kern = rows_bwd_kernel<T, TPR, NV, kBranch, kPre>;
  else kern = rows_fwd_kernel<T, TPR, NV, kBranch, kPre>;
  if (S::smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem) != cudaSuccess)
    return SWIN_ERR_CUDA;
  kern<<<ctas, S::threads, S::smem, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

template <typename T, int TPR, int NV>
int launch_rows(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st) {
  if (bwd) {
    if (branch && pre) return launch_one<T, TPR, NV, true, true, true>(a, ctas, st);
    if (branch) return launch_one<T, TPR, NV, true, true, false>(a, ctas, st);
    return launch_one<T, TPR, NV, true, false, true>(a, ctas, st);
  }
  if (branch && pre) return launch_one<T, TPR, NV, false, true, true>(a, ctas, st);
  if (branch) return launch_one<T, TPR, NV, false, true, false>(a, ctas, st);
  return launch_one<T, TPR, NV, false, false, true>(a, ctas, st);
}

template <typename T>
int launch_width(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st) {
  const Width wd = width_of(a.C);
  if (wd.tpr == 4) return launch_rows<T, 4, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 8) return launch_rows<T, 8, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 16) return launch_rows<T, 16, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 32 && wd.nv == 1) return launch_rows<T, 32, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 32) return launch_rows<T, 32, 2>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 128) return launch_rows<T, 128, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 256 && wd.nv == 1) return launch_rows<T, 256, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 256) return launch_rows<T, 256, 2>(a, bwd, branch, pre, ctas, st);
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
  const Split sp = split_rows(rows, r->channels, sms, true);
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
  const Split sp = split_rows(a.rows, a.C, sms, false);
  a.chunk = sp.chunk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return r->dtype == SWIN_BF16 ? launch_width<__nv_bfloat16>(a, false, false, true, sp.ctas, st)
                               : launch_width<float>(a, false, false, true, sp.ctas, st);
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
  const Split sp = split_rows(a.rows, a.C, sms, false);
  a.chunk = sp.chunk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return r->dtype == SWIN_BF16 ? launch_width<__nv_bfloat16>(a, false, true, pre, sp.ctas, st)
                               : launch_width<float>(a, false, true, pre, sp.ctas, st);
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
  const Split sp = split_rows(a.rows, a.C, sms, true);
  a.chunk = sp.chunk;
  if (want_pre || want_post) {
    if (!workspace || workspace_bytes < swin_attn_rows_workspace_bytes(r)) return SWIN_ERR_WORKSPACE;
    if (mis(workspace, 256)) return SWIN_ERR_ALIGNMENT;
    float *ws = static_cast<float *>(workspace);
    a.part_pre = want_pre ? ws : nullptr;
    a.part_post = want_post ? ws + (size_t)sp.ctas * 2 * a.C : nullptr;
  }
  if (a.rows) {
    rc = r->dtype == SWIN_BF16 ? launch_width<__nv_bfloat16>(a, true, branch, pre, sp.ctas, st)
                               : launch_width<float>(a, true, branch, pre, sp.ctas, st);
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
  c.kept = a.drop.scale * a.path.scale;
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
