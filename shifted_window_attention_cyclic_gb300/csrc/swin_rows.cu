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
// cancellation when the mean is large), and the results leave as whole sectors.
// The statistics are recomputed by the backward instead of stored.
// A row belongs to TPR threads, each holding NV vectors of 8 channels; the
// channels of a thread never change, so gamma, beta, scale and gate stay in
// registers and the column sums (the parameter gradients) accumulate there,
// per CTA, and are folded in a fixed order by a second kernel: no atomics, the
// same bits every run. All sums and statistics are fp32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
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
  bool wide;                    // fp32 outputs lie on 32-byte boundaries
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

// at byte `at` of a tensor. fp32: one 32-byte store where the tensor allows it;
// two of 16 bytes leave half of every sector to the other (join forward, fp32,
// 2 x 64 800 x 256: 130 us so, with halved loads too).
__device__ __forceinline__ void store8(void *base, int64_t at, const Raw<__nv_bfloat16> &r, bool) {
  *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(base) + at) = r.v;
}
__device__ __forceinline__ void store8(void *base, int64_t at, const Raw<float> &r, bool wide) {
  float4 *p = reinterpret_cast<float4 *>(static_cast<uint8_t *>(base) + at);
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(r.a.x), "f"(r.a.y),
                 "f"(r.a.z), "f"(r.a.w), "f"(r.b.x), "f"(r.b.y), "f"(r.b.z), "f"(r.b.w)
                 : "memory");
  } else {
    p[0] = r.a;
    p[1] = r.b;
  }
}

__device__ __forceinline__ void load8(const void *p, Raw<__nv_bfloat16> &r, bool) {
  r.v = *static_cast<const uint4 *>(p);
}
__device__ __forceinline__ void load8(const void *p, Raw<float> &r, bool wide) {
  if (wide) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r.a.x), "=f"(r.a.y), "=f"(r.a.z), "=f"(r.a.w), "=f"(r.b.x), "=f"(r.b.y), "=f"(r.b.z), "=f"(r.b.w)
                 : "l"(p)
                 : "memory");
  } else {
    r.a = static_cast<const float4 *>(p)[0];
    r.b = static_cast<const float4 *>(p)[1];
  }
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
// 16-byte asynchronous copies (cp.async); the bytes in flight do not depend on
// how many registers a warp's work takes. A bf16 vector is one copy, made by
// the thread that reads it. An fp32 vector is two: the lanes that share a row
// copy its pieces in order (each copy instruction whole sectors) and read their
// own two afterwards, so the ring is shared by a warp and needs its barriers.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int TPR, int NT, int NV, int kStages>
struct Ring {
  static constexpr int kThreads = TPR > 32 ? TPR : 256;
  static constexpr int kPieces = vec_bytes<T>() / 16;
  static constexpr int kStage = kThreads * NT * NV * vec_bytes<T>();
  static constexpr int W = TPR < 32 ? TPR : 32;  // lanes of a warp that share a row
  uint8_t *base;     // this thread's vector of slot 0
  uint32_t to[kPieces];  // and the pieces it copies, as shared addresses
  bool ok[NV][kPieces];  // pieces inside the row
  int lane_bytes;    // of a thread's first piece from its row's first byte

  __device__ __forceinline__ void init(uint8_t *smem, int lane, int C8) {
    const uint32_t s = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    const int t = threadIdx.x, w = t & ~31, l = t & 31;  // 16-byte chunks of fp32: 64 a warp, 2 l and 2 l + 1 a lane
    if constexpr (kPieces == 1) {
      base = smem + t * 16;
      to[0] = s + t * 16;
      lane_bytes = lane * 16;
    } else {
      base = smem + (w * 2 + swizzle(2 * l)) * 16;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) to[p] = s + (w * 2 + swizzle(l / W * 2 * W + p * W + l % W)) * 16;
      lane_bytes = (lane / 32 * 64 + lane % 32) * 16;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        ok[j][p] = j * TPR + (kPieces == 1 ? lane : lane / 32 * 32 + (p * W + lane % 32) / 2) < C8;
  }
  // keeps eight lanes' 32-byte reads free of bank conflicts (chunk 2 l + 1 follows or precedes 2 l)
  static __device__ __forceinline__ int swizzle(int chunk) { return chunk ^ ((chunk >> 3) & 1); }
  static __device__ __forceinline__ int slot(int t, int j) { return (t * NV + j) * kPieces * kThreads * 16; }
  // the stage after `stage` (stages are byte offsets)
  static __device__ __forceinline__ int next(int stage) { return stage == (kStages - 1) * kStage ? 0 : stage + kStage; }
  // a thread's pieces of vector j; `from`: byte of its first piece of the row's first vector (rows past the end: nothing
  // is read, zeros arrive)
  __device__ __forceinline__ void fetch(int stage, int t, int j, const void *tensor, int64_t from, bool row) const {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const bool there = row && ok[j][p];
      const int64_t at = there ? from + j * TPR * vec_bytes<T>() + p * W * 16 : 0;
      copy16(to[p] + stage + slot(t, j), static_cast<const uint8_t *>(tensor) + at, there);
    }
  }
  // before the slots of the stage read last are filled again
  __device__ __forceinline__ void before_fetch() const {
    if (kPieces > 1) __syncwarp();
  }
  // all but the newest N rows have arrived
  template <int N>
  __device__ __forceinline__ void arrived() const {
    copies_wait<N>();
    if (kPieces > 1) __syncwarp();
  }
  __device__ __forceinline__ void read(int stage, int t, int j, float2 (&f)[4]) const {
    const uint8_t *p = base + stage + slot(t, j);
    Raw<T> r;
    if constexpr (kPieces == 1) {
      r.v = *reinterpret_cast<const uint4 *>(p);
    } else {
      r.a = *reinterpret_cast<const float4 *>(p);
      r.b = *reinterpret_cast<const float4 *>(reinterpret_cast<const uint8_t *>(reinterpret_cast<uintptr_t>(p) ^ 16));
    }
    unpack(r, f);
  }
};

// ---- launch shapes ----------------------------------------------------------------
// One kernel's shape: TPR threads a row with NV vectors each, NT input tensors.
constexpr int block_of(int tpr) { return tpr > 32 ? tpr : 256; }

// Resident CTAs an SM (and the register bound that allows them). Backward: four
// column sums, two parameters and four rows of 8 channels are 80 registers a
// vector before any address, so 512 threads of one vector with 128 registers, or
// 256 of two. (640 threads with 96 registers spilled: 1-degree join backward
// 101 us against 91; 768 threads for the norm alone gained nothing.)
constexpr int blocks_per_sm(int tpr, int nv, bool bwd, bool branch) {
  return (bwd ? 512 / nv : nv == 2 ? 512 : branch ? 768 : 1024) / block_of(tpr) > 0
             ? (bwd ? 512 / nv : nv == 2 ? 512 : branch ? 768 : 1024) / block_of(tpr)
             : 1;
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
  static constexpr int blocks = blocks_per_sm(TPR, NV, kBwd, kBranch);
  static constexpr int tensors = kBwd ? 1 + (kPre ? 2 : 0) + (kBranch ? 1 : 0) : (kBranch ? 2 : 1);
  static constexpr int stage = threads * tensors * NV * vec_bytes<T>();
  static constexpr int ahead = rows_ahead(stage, blocks);
  static constexpr int flush = kBwd && TPR <= 32 ? threads * NV * 64 : 0;
  static constexpr int smem = (ahead + 1) * stage > flush ? (ahead + 1) * stage : flush;
  static_assert(smem <= 227 * 1024, "over a CTA's shared memory");
};

// The decisions of a thread's vectors of a row, one generator block each.
template <int NV>
__device__ __forceinline__ void draw_row(const Philox &ph, uint64_t vec, int step, uint4 (&bits)[NV]) {
  uint64_t at[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) at[j] = vec + (uint64_t)(j * step);
  ph.blocks(at, bits);
}

// ---- sums over a row ---------------------------------------------------------
// Sum of a float, or of a pair, over the TPR threads of a row. Rows of up to 32
// threads stay inside a warp; wider rows are the whole CTA and exchange one
// value per warp through one of two shared buffers (used in turn: one barrier
// per sum).
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float shuffle_xor(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ float2 shuffle_xor(float2 v, int o) { return make_float2(shuffle_xor(v.x, o), shuffle_xor(v.y, o)); }
template <int TPR, typename V>
__device__ __forceinline__ V row_sum(V v, float2 *xchg, int &turn) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v = add(v, shuffle_xor(v, o));
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    V *buf = reinterpret_cast<V *>(xchg + turn * W);
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

// Which of a CTA's rows a thread works on, and which channels.
struct Place {
  int lane, first, stride;  // thread of the row; its first row of the CTA's and the step to its next
};
template <int TPR>
__device__ __forceinline__ Place place() {
  constexpr int kWarps = block_of(TPR) / 32, RPW = TPR < 32 ? 32 / TPR : 1;  // rows a warp works on at once
  Place p;
  p.lane = TPR > 32 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  p.first = TPR > 32 ? 0 : (threadIdx.x >> 5) * RPW + (TPR < 32 ? (threadIdx.x & 31) / TPR : 0);
  p.stride = TPR > 32 ? 1 : kWarps * RPW;
  return p;
}
// Trips a thread's warp makes over `count` rows (the same for its whole warp).
template <int TPR>
__device__ __forceinline__ int trips(const Place &p, int count) {
  const int first = TPR < 32 ? p.first - (int)(threadIdx.x & 31) / TPR : p.first;
  return first < count ? (count - first + p.stride - 1) / p.stride : 0;
}

// ---- forward -----------------------------------------------------------------
// Norm of 1 179 648 rows x 256 bf16: 201 us, 6.0 TB/s (89 % of the measured copy
// rate): HBM. Join of 138 240 x 512 bf16 with both norms, gate, scale and dropout:
// 109 us, 5.2 TB/s (77 %): 16 warps an SM (128 registers) issue in 56 % of the
// cycles and wait on the two norms' sums in turn.
template <typename T, int TPR, int NV, bool kBranch, bool kPre>
__global__ void __launch_bounds__(block_of(TPR), blocks_per_sm(TPR, NV, false, kBranch)) rows_fwd_kernel(const RowArgs a) {
  using S = Shape<T, TPR, NV, false, kBranch, kPre>;
  constexpr int D = S::ahead, VB = vec_bytes<T>();
  using R = Ring<T, TPR, S::tensors, NV, D + 1>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 xchg[TPR > 32 ? 2 * (TPR / 32) : 1];
  int turn = 0;
  const Place pl = place<TPR>();
  const int C8 = a.C >> 3;
  const float inv = 1.0f / (float)a.C;
  R ring;
  ring.init(smem, pl.lane, C8);
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

  const int64_t first = (int64_t)blockIdx.x * a.chunk, last = min(first + a.chunk, a.rows);
  const int64_t step = (int64_t)pl.stride * C8;  // vectors from a thread's row to its next
  // one image of the CTA's rows at a time: the gate and the path decision change with it
  for (int64_t s = first; s < last;) {
    const int64_t b = s / a.tokens;
    const int count = (int)(min(last, (b + 1) * a.tokens) - s), n = trips<TPR>(pl, count);
    int64_t vec = (s + pl.first) * C8 + pl.lane;  // this row's first vector of the thread
    int64_t to = vec * VB;                        // and its byte, `step` vectors a row
    int64_t from = (s + pl.first) * C8 * VB + ring.lane_bytes;  // of its first piece of the row to fetch
    int ahead = pl.first;
    auto fetch = [&](int stage) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        ring.fetch(stage, 0, j, a.x, from, ahead < count);
        if constexpr (kBranch) ring.fetch(stage, 1, j, a.z, from, ahead < count);
      }
      copies_commit();
      ahead += pl.stride;
      from += step * VB;
    };
    int in = 0, out = 0;
#pragma unroll
    for (int k = 0; k < D; ++k, in += R::kStage) fetch(in);
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
    int row = pl.first;
#pragma unroll 1
    for (int k = 0; k < n; ++k, row += pl.stride, vec += step, to += step * VB) {
      ring.before_fetch();
      fetch(in);
      in = R::next(in);
      ring.template arrived<D>();
      const bool live = row < count;
      float2 v[NV][4];
#pragma unroll
      for (int j = 0; j < NV; ++j) ring.read(out, 0, j, v[j]);
      if constexpr (kBranch) {
        float2 u[NV][4];
#pragma unroll
        for (int j = 0; j < NV; ++j) ring.read(out, 1, j, u[j]);
        if (post) {
          if (a.post.kind == SWIN_NORM_LAYER) centre<NV>(u, row_sum<TPR>(sum_of<NV>(u), xchg, turn) * inv, ok);
          const float2 rstd = both(rsqrtf(fmaf(row_sum<TPR>(dot_of<NV>(u, u), xchg, turn), inv, a.post.eps)));
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) u[j][e] = mul(u[j][e], rstd);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
          for (int e = 0; e < 4; ++e) u[j][e] = fma(u[j][e], wg[j][e], wb[j][e]);
          if (a.drop.thr) {
            const uint4 bits = ph.block((uint64_t)(vec + j * TPR));
#pragma unroll
            for (int e = 0; e < 4; ++e) u[j][e] = kept(bits, e, a.drop.thr, u[j][e]);
          }
          if (path) {  // a dropped image's y is x
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j][e] = add(v[j][e], u[j][e]);
          }
          Raw<T> o;
          pack(v[j], o);
          if (ok[j] && live) store8(a.y, to + j * TPR * VB, o, a.wide);
          if constexpr (kPre) unpack(o, v[j]);  // h is the norm of y as stored
        }
      }
      out = R::next(out);
      if constexpr (kPre) {
        if (a.pre.kind == SWIN_NORM_LAYER) centre<NV>(v, row_sum<TPR>(sum_of<NV>(v), xchg, turn) * inv, ok);
        const float2 rstd = both(rsqrtf(fmaf(row_sum<TPR>(dot_of<NV>(v, v), xchg, turn), inv, a.pre.eps)));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          Raw<T> o;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] = fma(mul(v[j][e], rstd), gpre[j][e], bpre[j][e]);
          pack(v[j], o);
          if (ok[j] && live) store8(a.h, to + j * TPR * VB, o, a.wide);
        }
      }
    }
    copies_wait<0>();
    s += count;
  }
}

// ---- backward ----------------------------------------------------------------
// Sums the CTA's copies of this thread's channels of two column sums, writes
// them (one: dst[0, C), zero: dst[C, 2 C)) and clears them.
template <int TPR, int NV>
__device__ __forceinline__ void flush(float2 (&one)[NV][4], float2 (&zero)[NV][4], float *dst, int C8, float *buf) {
  constexpr int kThreads = block_of(TPR);
  const int lane = TPR > 32 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  auto put = [&](float *p, const float2 (&v)[4]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  };
  if constexpr (TPR > 32) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j * TPR + lane < C8) {
        put(dst + 8 * (j * TPR + lane), one[j]);
        put(dst + 8 * (C8 + j * TPR + lane), zero[j]);
      }
  } else {
    constexpr int G = kThreads / TPR, W = TPR * NV * 8;  // rows in flight, channels of a row (padded)
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float *p = buf + threadIdx.x / TPR * W + 8 * (j * TPR + lane);
      put(p, one[j]);
      put(p + G * W, zero[j]);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * W; c += kThreads) {
      const int h = c / W, ch = c % W;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < G; ++k) s += buf[(h * G + k) * W + ch];
      if (ch < 8 * C8) dst[h * 8 * C8 + ch] = s;
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) one[j][e] = zero[j][e] = make_float2(0.f, 0.f);
}

// Norm of 65 522 x 384 fp32 with the residual's gradient, parameters included: 66
// us, 6.1 TB/s (90 %): HBM. Join of 3 x 16 471 x 1024 bf16 (RMS, RMS, scale): 102 us,
// 5.9 TB/s (87 %). Join of 2 x 64 800 x 256 bf16 (LayerNorms, gate, scale, dropout,
// path): 84 us, 4.7 TB/s (70 %): 238 registers leave 8 warps an SM, which issue in
// 47 % of the cycles and wait on four rounds of row sums and on the generator.
template <typename T, int TPR, int NV, bool kBranch, bool kPre>
__global__ void __launch_bounds__(block_of(TPR), blocks_per_sm(TPR, NV, true, kBranch)) rows_bwd_kernel(const RowArgs a) {
  using S = Shape<T, TPR, NV, true, kBranch, kPre>;
  constexpr int D = S::ahead, VB = vec_bytes<T>();
  using R = Ring<T, TPR, S::tensors, NV, D + 1>;
  constexpr int tDy = 0, tY = 1, tDh = 2, tZ = kPre ? 3 : 1;  // tensors of a stage
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 xchg[TPR > 32 ? 2 * (TPR / 32) : 1];
  int turn = 0;
  const Place pl = place<TPR>();
  const int C8 = a.C >> 3;
  const float inv = 1.0f / (float)a.C;
  R ring;
  ring.init(smem, pl.lane, C8);
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
  const bool post = kBranch && a.post.kind != SWIN_NORM_NONE;
  const bool post_layer = kBranch && a.post.kind == SWIN_NORM_LAYER, pre_layer = kPre && a.pre.kind == SWIN_NORM_LAYER;

  const int64_t first = (int64_t)blockIdx.x * a.chunk, last = min(first + a.chunk, a.rows);
  const int64_t step = (int64_t)pl.stride * C8;
  for (int64_t s = first; s < last;) {
    const int64_t b = s / a.tokens;
    const int count = (int)(min(last, (b + 1) * a.tokens) - s), n = trips<TPR>(pl, count);
    int64_t vec = (s + pl.first) * C8 + pl.lane;
    int64_t to = vec * VB, from = (s + pl.first) * C8 * VB + ring.lane_bytes;
    int ahead = pl.first;
    auto fetch = [&](int stage) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (a.dy) ring.fetch(stage, tDy, j, a.dy, from, ahead < count);
        if constexpr (kPre) {
          ring.fetch(stage, tY, j, a.x, from, ahead < count);
          ring.fetch(stage, tDh, j, a.dh, from, ahead < count);
        }
        if constexpr (kBranch)
          if (a.z) ring.fetch(stage, tZ, j, a.z, from, ahead < count);
      }
      copies_commit();
      ahead += pl.stride;
      from += step * VB;
    };
    int in = 0, out = 0;
#pragma unroll
    for (int k = 0; k < D; ++k, in += R::kStage) fetch(in);
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
    int row = pl.first;
    // Vectors past a row's end and rows past the last arrive as zeros and stay
    // zeros (u, dh, g), so they add nothing to any sum.
#pragma unroll 1
    for (int k = 0; k < n; ++k, row += pl.stride, vec += step, to += step * VB) {
      ring.before_fetch();
      fetch(in);
      in = R::next(in);
      uint4 bits[NV];  // drawn together here, where no row waits for them yet (1-degree: 87 us, 89 us at their use)
      if (kBranch && a.drop.thr) draw_row(ph, vec, TPR, bits);
      ring.template arrived<D>();
      const bool live = row < count;
      // both rows' statistics, in two rounds of sums
      float2 y[NV][4], z[NV][4];
      float y_rstd = 1.f, z_rstd = 1.f;
      if constexpr (kPre) {
#pragma unroll
        for (int j = 0; j < NV; ++j) ring.read(out, tY, j, y[j]);
      }
      if constexpr (kBranch) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (a.z && path) {
            ring.read(out, tZ, j, z[j]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) z[j][e] = make_float2(0.f, 0.f);
          }
        }
      }
      if constexpr (kPre && kBranch) {
        if (post) {
          if (pre_layer || post_layer) {
            const float2 m = row_sum<TPR>(make_float2(sum_of<NV>(y), sum_of<NV>(z)), xchg, turn);
            if (pre_layer) centre<NV>(y, m.x * inv, ok);
            if (post_layer) centre<NV>(z, m.y * inv, ok);
          }
          const float2 q = row_sum<TPR>(make_float2(dot_of<NV>(y, y), dot_of<NV>(z, z)), xchg, turn);
          y_rstd = rsqrtf(fmaf(q.x, inv, a.pre.eps));
          z_rstd = rsqrtf(fmaf(q.y, inv, a.post.eps));
        }
      }
      if constexpr (kPre)
        if (!kBranch || !post) {
          if (pre_layer) centre<NV>(y, row_sum<TPR>(sum_of<NV>(y), xchg, turn) * inv, ok);
          y_rstd = rsqrtf(fmaf(row_sum<TPR>(dot_of<NV>(y, y), xchg, turn), inv, a.pre.eps));
        }
      if constexpr (kBranch && !kPre)
        if (post) {
          if (post_layer) centre<NV>(z, row_sum<TPR>(sum_of<NV>(z), xchg, turn) * inv, ok);
          z_rstd = rsqrtf(fmaf(row_sum<TPR>(dot_of<NV>(z, z), xchg, turn), inv, a.post.eps));
        }
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
        float2 dh[NV][4];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          ring.read(out, tDh, j, dh[j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[j][e] = mul(y[j][e], both(y_rstd));
            a1[j][e] = fma(dh[j][e], y[j][e], a1[j][e]);
            a0[j][e] = add(a0[j][e], dh[j][e]);
            dh[j][e] = mul(dh[j][e], gpre[j][e]);
          }
        }
        float2 c = make_float2(dot_of<NV>(dh, y), 0.f);
        if (pre_layer) {
          c.y = sum_of<NV>(dh);
          c = row_sum<TPR>(c, xchg, turn);
        } else {
          c.x = row_sum<TPR>(c.x, xchg, turn);
        }
        const float2 c1 = both(-c.x * inv);
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float2 c0 = both(ok[j] ? -c.y * inv : 0.f);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            g[j][e] = fma(both(y_rstd), add(dh[j][e], fma(y[j][e], c1, c0)), g[j][e]);
        }
      }
      out = R::next(out);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        Raw<T> o;
        pack(g[j], o);
        if (ok[j] && live) store8(a.dx, to + j * TPR * VB, o, a.wide);
      }
      if constexpr (kBranch) {
        if (path) {
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            if (post) {
#pragma unroll
              for (int e = 0; e < 4; ++e) z[j][e] = mul(z[j][e], both(z_rstd));
            }
            if (a.drop.thr) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                g[j][e] = kept(bits[j], e, a.drop.thr, g[j][e]);
                // what was dropped takes no part, were it infinite (a row's norm has it in its statistics anyway)
                if (!post) z[j][e] = kept(bits[j], e, a.drop.thr, z[j][e]);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              b1[j][e] = fma(g[j][e], z[j][e], b1[j][e]);
              b0[j][e] = add(b0[j][e], g[j][e]);
              g[j][e] = mul(g[j][e], w[j][e]);
            }
          }
          if (post) {
            float2 c = make_float2(dot_of<NV>(g, z), 0.f);
            if (post_layer) {
              c.y = sum_of<NV>(g);
              c = row_sum<TPR>(c, xchg, turn);
            } else {
              c.x = row_sum<TPR>(c.x, xchg, turn);
            }
            const float2 c1 = both(-c.x * inv), c0 = both(-c.y * inv);
#pragma unroll
            for (int j = 0; j < NV; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) g[j][e] = mul(both(z_rstd), add(g[j][e], fma(z[j][e], c1, c0)));
          }
        } else {  // a dropped image: no gradient reaches z
#pragma unroll
          for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) g[j][e] = make_float2(0.f, 0.f);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          Raw<T> o;
          pack(g[j], o);
          if (ok[j] && live) store8(a.dz, to + j * TPR * VB, o, a.wide);
        }
      }
    }
    copies_wait<0>();
    s += count;
    // with a gate the sums are kept per image: slot CTA + image (a CTA's next
    // image takes its next slot, the next CTA's first is one further)
    if constexpr (kBranch)
      if (a.part_post && (a.gate || s == last)) {
        float *dst = a.part_post + ((int64_t)blockIdx.x + (a.gate ? b : 0)) * 2 * a.C;
        flush<TPR, NV>(b1, b0, dst, C8, reinterpret_cast<float *>(smem));
        if (TPR <= 32) __syncthreads();  // the ring takes the buffer again
      }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (kPre)
    if (a.part_pre) {
      float *dst = a.part_pre + (int64_t)blockIdx.x * 2 * a.C;
      flush<TPR, NV>(a1, a0, dst, C8, reinterpret_cast<float *>(smem));
    }
}

// ---- parameter gradients from the column sums ----------------------------------
struct ColArgs {
  int64_t tokens, chunk;
  int images, C, ctas;  // ctas: slots of each CTA sum (0: no rows)
  bool post_norm;
  float kept;  // what kept values are multiplied by (left out of the join's sums)
  const float *part_pre, *part_post;
  const float *scale, *gate, *gamma, *beta;  // gamma, beta: the post norm's
  float *dpre_gamma, *dpre_beta, *dpost_gamma, *dpost_beta, *dscale, *dgate;
  float *groups;  // [gridDim.y][2][C] gate-weighted sums of each group of images, where there are several
};

constexpr int kColLanes = 32, kGroupImages = 256, kFewImages = 4;

struct Sums {
  float one, zero;  // of the terms with xhat, and of those without
};

// Adds up the lanes of a block (32 channels x kColLanes) in a fixed order: warp y
// sums channel y, so thread (0, y) has the result.
__device__ __forceinline__ Sums lane_sum(Sums v, float2 (&buf)[kColLanes][33]) {
  __syncthreads();
  buf[threadIdx.y][threadIdx.x] = make_float2(v.one, v.zero);
  __syncthreads();
  float2 s = buf[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s = add(s, shuffle_xor(s, o));
  return {s.x, s.y};
}

// Slots s0 ... s1 of channel c, every `step`th.
__device__ __forceinline__ Sums slot_sum(const float *part, int s0, int s1, int step, int C, int c) {
  Sums v = {0.f, 0.f};
  const float *p = part + (int64_t)s0 * 2 * C + c;
#pragma unroll 8
  for (int s = s0; s <= s1; s += step, p += (int64_t)step * 2 * C) {
    v.one += p[0];
    v.zero += p[C];
  }
  return v;
}

// Block (tile, group, 0 or 1): 32 channels. z = 0: the pre norm's sums over all
// rows. z = 1: the join's, and with a gate each group its images: their gate
// gradients and their gate-weighted sum. The pair (CTA r, image b) has slot
// r + b, so image b owns the slots from its first row's CTA to its last row's.
// A few images share the lanes; many take a lane each. Latency bound: 7 us with
// cold caches, 3 to 6 us behind the row kernel, whose sums lie in L2.
__global__ void __launch_bounds__(32 * kColLanes) columns_kernel(const ColArgs a) {
  static_assert(kColLanes == 32, "a warp sums the lanes of a channel");
  // launched while the row kernel's last CTAs still run: their sums are there after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float2 buf[kColLanes][33];
  const int tile = blockIdx.x * 32, lane = threadIdx.y;
  const int cc = min(tile + (int)threadIdx.x, a.C - 1);  // the channel this thread sums
  const int c = tile + (int)threadIdx.y;                 // the channel whose result its warp gets
  const bool own = threadIdx.x == 0 && c < a.C;
  if (blockIdx.z == 0) {
    if (blockIdx.y > 0 || !(a.dpre_gamma || a.dpre_beta)) return;
    const Sums v = lane_sum(slot_sum(a.part_pre, lane, a.ctas - 1, kColLanes, a.C, cc), buf);
    if (own && a.dpre_gamma) a.dpre_gamma[c] = v.one;
    if (own && a.dpre_beta) a.dpre_beta[c] = v.zero;
    return;
  }
  if (!a.dpost_gamma && !a.dpost_beta && !a.dscale && !a.dgate) return;
  auto at = [&](const float *p, int ch, float none) { return p ? p[min(ch, a.C - 1)] : none; };
  const float *gamma = a.post_norm ? a.gamma : nullptr, *beta = a.post_norm ? a.beta : nullptr;
  Sums all = {0.f, 0.f};
  if (!a.gate) {
    all = lane_sum(slot_sum(a.part_post, lane, a.ctas - 1, kColLanes, a.C, cc), buf);
  } else {
    const int tokens = (int)a.tokens, chunk = (int)a.chunk;  // both, and all rows, below 2^31
    const int b0 = blockIdx.y * kGroupImages, b1 = min(b0 + kGroupImages, a.images);
    auto slots = [&](int b, int &s0, int &s1) {
      s0 = tokens * b / chunk + b;
      s1 = a.ctas ? (tokens * (b + 1) - 1) / chunk + b : s0 - 1;
    };
    auto image = [&](int b, int ch, const Sums &v, bool store) {
      if (ch >= a.C) return;
      const float g = a.gate[(int64_t)b * a.C + ch];
      all.one = fmaf(g, v.one, all.one);
      all.zero = fmaf(g, v.zero, all.zero);
      if (a.dgate && store)
        a.dgate[(int64_t)b * a.C + ch] =
            a.kept * at(a.scale, ch, 1.f) * fmaf(at(gamma, ch, 1.f), v.one, at(beta, ch, 0.f) * v.zero);
    };
    if (b1 - b0 <= kFewImages) {
      Sums v[kFewImages];
#pragma unroll
      for (int k = 0; k < kFewImages; ++k) {
        int s0 = 0, s1 = -1;
        if (b0 + k < b1) slots(b0 + k, s0, s1);
        v[k] = slot_sum(a.part_post, s0 + lane, s1, kColLanes, a.C, cc);
      }
#pragma unroll
      for (int k = 0; k < kFewImages; ++k)
        if (b0 + k < b1) image(b0 + k, c, lane_sum(v[k], buf), threadIdx.x == 0);
    } else {
      for (int b = b0 + lane; b < b1; b += kColLanes) {
        int s0, s1;
        slots(b, s0, s1);
        image(b, tile + (int)threadIdx.x, slot_sum(a.part_post, s0, s1, 1, a.C, cc), true);
      }
      all = lane_sum(all, buf);
    }
  }
  if (!own) return;
  if (a.groups) {
    a.groups[(int64_t)blockIdx.y * 2 * a.C + c] = all.one;
    a.groups[(int64_t)blockIdx.y * 2 * a.C + a.C + c] = all.zero;
  } else {
    if (a.dpost_gamma) a.dpost_gamma[c] = a.kept * at(a.scale, c, 1.f) * all.one;
    if (a.dpost_beta) a.dpost_beta[c] = a.kept * at(a.scale, c, 1.f) * all.zero;
    if (a.dscale) a.dscale[c] = a.kept * fmaf(at(gamma, c, 1.f), all.one, at(beta, c, 0.f) * all.zero);
  }
}

// ---- dropout -------------------------------------------------------------------
// Element i keeps iff decision i / span does. kMode 0: span 1, one block per
// 8-element vector; 1: span a multiple of 8, one decision per vector; 2: any
// other span, one decision per element. 302 M bf16 elements, span 1: 187 us, 6.4
// TB/s (95 % of the measured copy rate): HBM; the generator's wide multiplies fill
// 57 % of their pipe.
template <typename T, int kMode>
__global__ void __launch_bounds__(256) dropout_kernel(const T *x, T *y, int64_t n, int64_t span, Drop d, bool wide) {
  Philox ph;
  ph.init(d);
  const int64_t nvec = (n + 7) >> 3;
  for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < nvec; v += (int64_t)gridDim.x * 256) {
    const int64_t i0 = v * 8;
    uint4 bits = make_uint4(0u, 0u, 0u, 0u);
    if (kMode == 0) bits = ph.block((uint64_t)v);
    if (kMode == 1) {  // (32-bit division: a quarter of the long one's work)
      const uint64_t i = nvec <= UINT32_MAX ? (uint32_t)v / (uint32_t)min(span >> 3, (int64_t)UINT32_MAX) : v / (span >> 3);
      if (keep_one(ph, i, d.thr)) bits = make_uint4(~0u, ~0u, ~0u, ~0u);
    }
    if (i0 + 8 <= n) {
      Raw<T> in;
      load8(x + i0, in, wide);
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
      store8(y, i0 * (int64_t)sizeof(T), out, wide);
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

// Threads per row and vectors per thread: the fewest that hold the row. Two
// vectors a thread where a warp holds rows: more rows share a warp's shuffles
// and addresses than with one (256 channels: norm of 1 179 648 rows 201 us
// against 210, join 54 against 58, its backward 89 against 91). From 513 channels
// on a row is a CTA's: one vector a thread up to 2048 (two warps a row for 512
// channels gained nothing: join forward 109 us against 107), two above.
Width width_of(int C) {
  const int c8 = C >> 3;
  if (c8 <= 4) return {4, 1};
  if (c8 <= 8) return {4, 2};
  if (c8 <= 16) return {8, 2};
  if (c8 <= 32) return {16, 2};
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
Split split_rows(int64_t rows, int C, int sms, bool bwd, bool branch) {
  const Width wd = width_of(C);
  const int64_t at_once = wd.tpr > 32 ? 1 : 256 / wd.tpr;
  const int64_t groups = (rows + at_once - 1) / at_once;
  const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)sms * blocks_per_sm(wd.tpr, wd.nv, bwd, branch)));
  int64_t chunk = (rows + ctas - 1) / ctas;
  chunk = std::max<int64_t>(1, (chunk + at_once - 1) / at_once * at_once);
  return {chunk, (int)((rows + chunk - 1) / chunk)};
}

// SMs of the current device (asked once per device: the calls are short).
int sm_count(int *sms) {
  static std::atomic<int> known[64];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return SWIN_ERR_CUDA;
  if (dev < 64 && (*sms = known[dev].load(std::memory_order_relaxed)) > 0) return SWIN_OK;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return SWIN_ERR_CUDA;
  if (dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
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
  if (wd.tpr == 4 && wd.nv == 1) return launch_rows<T, 4, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 4) return launch_rows<T, 4, 2>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 8) return launch_rows<T, 8, 2>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 16) return launch_rows<T, 16, 2>(a, bwd, branch, pre, ctas, st);
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

// Column sums in the workspace: of the pre norm [ctas], of the join [ctas + images], of image groups.
int64_t join_slots(int ctas, int64_t images) { return (int64_t)ctas + std::max<int64_t>(images, 1); }
int64_t image_groups(int64_t images) { return std::max<int64_t>(1, (images + kGroupImages - 1) / kGroupImages); }

}  // namespace
}  // namespace swin

using namespace swin;

extern "C" {

size_t swin_attn_rows_workspace_bytes(const swin_attn_rows *r) {
  int64_t rows = 0;
  size_t bytes = 0;
  int sms = 0;
  if (check_rows(r, &rows, &bytes) || sm_count(&sms)) return 0;
  const Split sp = split_rows(rows, r->channels, sms, true, true);
  const size_t slots = (size_t)(sp.ctas + join_slots(sp.ctas, r->images) + image_groups(r->images));
  const size_t need = slots * 2 * r->channels * sizeof(float);
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
  a.wide = !mis(h, 32);
  a.tokens = a.rows;
  a.images = 1;
  a.C = r->channels;
  a.path.scale = a.drop.scale = 1.f;
  const Split sp = split_rows(a.rows, a.C, sms, false, false);
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
  a.wide = !mis(y, 32) && !mis(h, 32);
  a.scale = join->scale;
  a.gate = join->gate;
  a.tokens = r->tokens;
  a.images = (int)r->images;
  a.C = r->channels;
  const Split sp = split_rows(a.rows, a.C, sms, false, true);
  a.chunk = sp.chunk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return r->dtype == SWIN_BF16 ? launch_width<__nv_bfloat16>(a, false, true, pre, sp.ctas, st)
                               : launch_width<float>(a, false, true, pre, sp.ctas, st);
}

}  // extern "C"

namespace {

// As a programmatic dependent of the kernel before it in the stream: its launch
// overlaps that kernel's end (the fold took 10 us behind a backward of 80 us).
int launch_columns(const ColArgs &c, int tiles, unsigned groups, cudaStream_t st) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(tiles, groups, 2);
  cfg.blockDim = dim3(32, kColLanes);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, columns_kernel, c) == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

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
  const int64_t groups = a.gate && want_post ? image_groups(a.images) : 1;
  if (groups > 65535) return SWIN_ERR_UNSUPPORTED;  // (a grid's y)
  const Split sp = split_rows(a.rows, a.C, sms, true, true);
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
  const int tiles = (a.C + 31) / 32;
  if (groups > 1) c.groups = a.part_post + join_slots(sp.ctas, a.images) * 2 * a.C;
  if ((rc = launch_columns(c, tiles, (unsigned)groups, st))) return rc;
  if (groups > 1) {  // the groups' sums are what a join without a gate would have left
    c.part_post = c.groups;
    c.ctas = (int)groups;
    c.gate = nullptr;
    c.groups = c.dgate = c.dpre_gamma = c.dpre_beta = nullptr;
    rc = launch_columns(c, tiles, 1, st);
  }
  return rc;
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
  a.wide = !mis(dx, 32);
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
  a.wide = !mis(dx, 32) && !mis(dz, 32);
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
    if (mode == 0) dropout_kernel<__nv_bfloat16, 0><<<blocks, 256, 0, st>>>(p, q, n, span, d, !mis(x, 32) && !mis(y, 32));
    else if (mode == 1) dropout_kernel<__nv_bfloat16, 1><<<blocks, 256, 0, st>>>(p, q, n, span, d, !mis(x, 32) && !mis(y, 32));
    else dropout_kernel<__nv_bfloat16, 2><<<blocks, 256, 0, st>>>(p, q, n, span, d, !mis(x, 32) && !mis(y, 32));
  } else {
    const float *p = static_cast<const float *>(x);
    float *q = static_cast<float *>(y);
    if (mode == 0) dropout_kernel<float, 0><<<blocks, 256, 0, st>>>(p, q, n, span, d, !mis(x, 32) && !mis(y, 32));
    else if (mode == 1) dropout_kernel<float, 1><<<blocks, 256, 0, st>>>(p, q, n, span, d, !mis(x, 32) && !mis(y, 32));
    else dropout_kernel<float, 2><<<blocks, 256, 0, st>>>(p, q, n, span, d, !mis(x, 32) && !mis(y, 32));
  }
  return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

}  // extern "C"
