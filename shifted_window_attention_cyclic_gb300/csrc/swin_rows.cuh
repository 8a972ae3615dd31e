// swin_rows.cuh -- the row kernels of swin_rows.cu: norm and residual join,
// forward and backward. Included by one translation unit per activation type.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "swin_common.cuh"
#include "swin_philox.cuh"
#include "swin_vec8.cuh"

namespace swin {
namespace rows {

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

// Threads of a row: TPR, or where a row is a CTA of as many warps as it needs, the CTA's.
template <int TPR, bool kFull>
__device__ __forceinline__ int threads_of_row() { return kFull ? TPR : (int)blockDim.x; }

template <typename T, int TPR, bool kFull, int NT, int NV, int kStages>
struct Ring {
  static constexpr int kThreads = TPR > 32 ? TPR : 256;  // a wide row's CTA may have fewer
  static constexpr int kPieces = vec_bytes<T>() / 16;
  static constexpr int kStage = kThreads * NT * NV * vec_bytes<T>();
  static constexpr int W = TPR < 32 ? TPR : 32;  // lanes of a warp that share a row
  uint8_t *base;     // this thread's vector of slot 0
  uint32_t to[kPieces];  // and the pieces it copies, as shared addresses
  bool ok[NV][kPieces];  // pieces inside the row
  int lane_bytes;    // of a thread's first piece from its row's first byte
  int tpr;           // threads of a row

  __device__ __forceinline__ void init(uint8_t *smem, int lane, int C8) {
    tpr = threads_of_row<TPR, kFull>();
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
        ok[j][p] = j * tpr + (kPieces == 1 ? lane : lane / 32 * 32 + (p * W + lane % 32) / 2) < C8;
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
      const int64_t at = there ? from + j * tpr * vec_bytes<T>() + p * W * 16 : 0;
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

// Resident CTAs an SM: the register bound of a kernel. Backward: four column
// sums, two parameters and four rows of 8 channels are 80 registers a vector
// before any address, so 512 threads of one vector with 128 registers, or 256
// of two or three. (640 threads with 96 registers spilled: 1-degree join backward
// 101 us against 91; 768 threads for the norm alone gained nothing.) A row that
// is a CTA's waits in every round of its sums, so two CTAs an SM pay more than
// registers: the norm alone in 128 (75 M bf16 elements in 4096 channels 126 -> 107
// us, in 3584 138 -> 109), and a CTA of 160 threads, 2049 to 2560 bf16 channels,
// in 168 (10 warps are three on a scheduler), of which both norms' join spills
// 24: 2056 channels, norm 221 -> 139 us, join without a norm after it 213 -> 117,
// with both norms and dropout 433 -> 321.
constexpr int blocks_per_sm(int tpr, int nv, bool bwd, bool branch) {
  const int threads = bwd ? (tpr == 160 ? 320 : nv == 1 || (tpr == 256 && !branch) ? 512 : 256) : nv == 3 ? (branch ? 256 : 512) : nv == 2 ? 512 : branch ? 768 : 1024;
  return threads > block_of(tpr) ? threads / block_of(tpr) : 1;
}

// Rows ahead: 64 KB in flight on an SM cover HBM's latency at its rate (about
// 1 us at 45 GB/s a SM), as far as 200 KB of shared memory hold the ring.
constexpr int rows_ahead(int stage_bytes, int blocks) {
  int d = (65536 + blocks * stage_bytes - 1) / (blocks * stage_bytes);
  const int most = 200 * 1024 / blocks / stage_bytes - 1;
  d = d > most ? most : d;
  return d < 0 ? 0 : d > 7 ? 7 : d;
}

constexpr int tensors_of(bool bwd, bool branch, bool pre) {
  return bwd ? 1 + (pre ? 2 : 0) + (branch ? 1 : 0) : branch ? 2 : 1;
}
constexpr int stage_of(int tpr, int nv, bool bwd, bool branch, bool pre, int bytes) {
  return block_of(tpr) * tensors_of(bwd, branch, pre) * nv * 8 * bytes;
}
// Dynamic shared memory of a CTA: the ring, which the flush of the column sums uses again.
constexpr int smem_of(int tpr, int nv, bool bwd, bool branch, bool pre, int bytes) {
  const int stage = stage_of(tpr, nv, bwd, branch, pre, bytes);
  const int ring = (rows_ahead(stage, blocks_per_sm(tpr, nv, bwd, branch)) + 1) * stage;
  const int flush = bwd && tpr <= 32 ? block_of(tpr) * nv * 64 : 0;
  return ring > flush ? ring : flush;
}

template <typename T, int TPR, int NV, bool kBwd, bool kBranch, bool kPre>
struct Shape {
  static constexpr int threads = block_of(TPR);  // at most
  static constexpr int tensors = tensors_of(kBwd, kBranch, kPre);
  static constexpr int ahead = rows_ahead(stage_of(TPR, NV, kBwd, kBranch, kPre, sizeof(T)), blocks_per_sm(TPR, NV, kBwd, kBranch));
  static constexpr int smem = smem_of(TPR, NV, kBwd, kBranch, kPre, sizeof(T));
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
// threads stay inside a warp; wider rows are the whole CTA (TPR threads at most,
// as many warps as the row needs) and exchange one value per warp through one of two shared buffers (used in turn: one barrier
// per sum).
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float shuffle_xor(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ float2 shuffle_xor(float2 v, int o) { return make_float2(shuffle_xor(v.x, o), shuffle_xor(v.y, o)); }
template <int TPR, bool kFull, typename V>
__device__ __forceinline__ V row_sum(V v, float2 *xchg, int &turn) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v = add(v, shuffle_xor(v, o));
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;  // at most
    const int warps = threads_of_row<TPR, kFull>() >> 5;
    V *buf = reinterpret_cast<V *>(xchg + turn * W);
    turn ^= 1;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
    if (warps == W) {
#pragma unroll
      for (int w = 1; w < W; ++w) v = add(v, buf[w]);
    } else {
#pragma unroll
      for (int w = 1; w < W; ++w)
        if (w < warps) v = add(v, buf[w]);
    }
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
template <typename T, int TPR, bool kFull, int NV, bool kBranch, bool kPre>
__global__ void __launch_bounds__(block_of(TPR), blocks_per_sm(TPR, NV, false, kBranch)) rows_fwd_kernel(const RowArgs a) {
  using S = Shape<T, TPR, NV, false, kBranch, kPre>;
  const int tpr = threads_of_row<TPR, kFull>();
  constexpr int D = S::ahead, VB = vec_bytes<T>();
  using R = Ring<T, TPR, kFull, S::tensors, NV, D + 1>;
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
    ok[j] = j * tpr + pl.lane < C8;
    if constexpr (kPre) {
      load_param(a.pre.gamma, j * tpr + pl.lane, ok[j], 1.f, gpre[j]);
      load_param(a.pre.beta, j * tpr + pl.lane, ok[j], 0.f, bpre[j]);
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
        load_param(a.scale, j * tpr + pl.lane, ok[j], 1.f, wg[j]);
        load_param(a.gate ? a.gate + b * a.C : nullptr, j * tpr + pl.lane, ok[j], 1.f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) wb[j][e] = wg[j][e] = mul(mul(wg[j][e], t[e]), both(c));
        load_param(a.post.gamma, j * tpr + pl.lane, ok[j] && post, 1.f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) wg[j][e] = mul(wg[j][e], t[e]);
        load_param(a.post.beta, j * tpr + pl.lane, ok[j] && post, 0.f, t);
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
          if (a.post.kind == SWIN_NORM_LAYER) centre<NV>(u, row_sum<TPR, kFull>(sum_of<NV>(u), xchg, turn) * inv, ok);
          const float2 rstd = both(rsqrtf(fmaf(row_sum<TPR, kFull>(dot_of<NV>(u, u), xchg, turn), inv, a.post.eps)));
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
            const uint4 bits = ph.block((uint64_t)(vec + j * tpr));
#pragma unroll
            for (int e = 0; e < 4; ++e) u[j][e] = kept(bits, e, a.drop.thr, u[j][e]);
          }
          if (path) {  // a dropped image's y is x
#pragma unroll
            for (int e = 0; e < 4; ++e) v[j][e] = add(v[j][e], u[j][e]);
          }
          Raw<T> o;
          pack(v[j], o);
          if (ok[j] && live) store8(a.y, to + j * tpr * VB, o, a.wide);
          if constexpr (kPre) unpack(o, v[j]);  // h is the norm of y as stored
        }
      }
      out = R::next(out);
      if constexpr (kPre) {
        if (a.pre.kind == SWIN_NORM_LAYER) centre<NV>(v, row_sum<TPR, kFull>(sum_of<NV>(v), xchg, turn) * inv, ok);
        const float2 rstd = both(rsqrtf(fmaf(row_sum<TPR, kFull>(dot_of<NV>(v, v), xchg, turn), inv, a.pre.eps)));
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          Raw<T> o;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] = fma(mul(v[j][e], rstd), gpre[j][e], bpre[j][e]);
          pack(v[j], o);
          if (ok[j] && live) store8(a.h, to + j * tpr * VB, o, a.wide);
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
template <int TPR, bool kFull, int NV>
__device__ __forceinline__ void flush(float2 (&one)[NV][4], float2 (&zero)[NV][4], float *dst, int C8, float *buf) {
  constexpr int kThreads = block_of(TPR);
  const int tpr = threads_of_row<TPR, kFull>();
  const int lane = TPR > 32 ? (int)threadIdx.x : (int)threadIdx.x % TPR;
  auto put = [&](float *p, const float2 (&v)[4]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  };
  if constexpr (TPR > 32) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (j * tpr + lane < C8) {
        put(dst + 8 * (j * tpr + lane), one[j]);
        put(dst + 8 * (C8 + j * tpr + lane), zero[j]);
      }
  } else {
    constexpr int G = kThreads / TPR, W = TPR * NV * 8;  // rows in flight, channels of a row (padded)
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float *p = buf + threadIdx.x / TPR * W + 8 * (j * tpr + lane);
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
template <typename T, int TPR, bool kFull, int NV, bool kBranch, bool kPre>
__global__ void __launch_bounds__(block_of(TPR), blocks_per_sm(TPR, NV, true, kBranch)) rows_bwd_kernel(const RowArgs a) {
  using S = Shape<T, TPR, NV, true, kBranch, kPre>;
  const int tpr = threads_of_row<TPR, kFull>();
  constexpr int D = S::ahead, VB = vec_bytes<T>();
  using R = Ring<T, TPR, kFull, S::tensors, NV, D + 1>;
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
    ok[j] = j * tpr + pl.lane < C8;
    if constexpr (kPre) load_param(a.pre.gamma, j * tpr + pl.lane, ok[j], 1.f, gpre[j]);
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
        load_param(a.scale, j * tpr + pl.lane, ok[j], 1.f, w[j]);
        load_param(a.gate ? a.gate + b * a.C : nullptr, j * tpr + pl.lane, ok[j], 1.f, t);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[j][e] = mul(mul(w[j][e], t[e]), both(c));
        load_param(a.post.gamma, j * tpr + pl.lane, ok[j] && post, 1.f, t);
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
      if (kBranch && a.drop.thr) draw_row(ph, vec, tpr, bits);
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
            const float2 m = row_sum<TPR, kFull>(make_float2(sum_of<NV>(y), sum_of<NV>(z)), xchg, turn);
            if (pre_layer) centre<NV>(y, m.x * inv, ok);
            if (post_layer) centre<NV>(z, m.y * inv, ok);
          }
          const float2 q = row_sum<TPR, kFull>(make_float2(dot_of<NV>(y, y), dot_of<NV>(z, z)), xchg, turn);
          y_rstd = rsqrtf(fmaf(q.x, inv, a.pre.eps));
          z_rstd = rsqrtf(fmaf(q.y, inv, a.post.eps));
        }
      }
      if constexpr (kPre)
        if (!kBranch || !post) {
          if (pre_layer) centre<NV>(y, row_sum<TPR, kFull>(sum_of<NV>(y), xchg, turn) * inv, ok);
          y_rstd = rsqrtf(fmaf(row_sum<TPR, kFull>(dot_of<NV>(y, y), xchg, turn), inv, a.pre.eps));
        }
      if constexpr (kBranch && !kPre)
        if (post) {
          if (post_layer) centre<NV>(z, row_sum<TPR, kFull>(sum_of<NV>(z), xchg, turn) * inv, ok);
          z_rstd = rsqrtf(fmaf(row_sum<TPR, kFull>(dot_of<NV>(z, z), xchg, turn), inv, a.post.eps));
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
          c = row_sum<TPR, kFull>(c, xchg, turn);
        } else {
          c.x = row_sum<TPR, kFull>(c.x, xchg, turn);
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
        if (ok[j] && live) store8(a.dx, to + j * tpr * VB, o, a.wide);
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
              c = row_sum<TPR, kFull>(c, xchg, turn);
            } else {
              c.x = row_sum<TPR, kFull>(c.x, xchg, turn);
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
          if (ok[j] && live) store8(a.dz, to + j * tpr * VB, o, a.wide);
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
        flush<TPR, kFull, NV>(b1, b0, dst, C8, reinterpret_cast<float *>(smem));
        if (TPR <= 32) __syncthreads();  // the ring takes the buffer again
      }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (kPre)
    if (a.part_pre) {
      float *dst = a.part_pre + (int64_t)blockIdx.x * 2 * a.C;
      flush<TPR, kFull, NV>(a1, a0, dst, C8, reinterpret_cast<float *>(smem));
    }
}

// ---- launch shapes of a call --------------------------------------------------------
struct Width {
  int tpr, nv;
};

// Threads per row and vectors per thread: the fewest that hold the row. Several
// vectors a thread where a warp holds rows: more rows share a warp's shuffles
// and addresses (256 channels, two against one: norm of 1 179 648 rows 201 us
// against 210, join 54 against 58, its backward 89 against 91), and few lanes idle
// (three, of 75 M elements: 384 channels, join 103 us against 128 with two,
// norm backward 103 against 115; 768 channels, join 108 us against 142 with a
// CTA's three warps a row). Above, a row is a CTA's, with as many warps as it
// needs, one vector a thread up to 2048 channels, two from there. (fp32 rows of 2049
// to 2560 channels stay with the bound of 256 threads: twice the bytes a row keep
// HBM busy, and the join backward with both norms took 246 us against 232 in 168
// registers.) Of the backward
// with both norms three vectors spill: they pay between 129 and 192 and between
// 257 and 384 channels, where a third of the lanes would idle.
inline Width width_of(int C, bool both_backward, bool bf16) {
  const int c8 = C >> 3;
  if (c8 <= 2) return {2, 1};
  if (c8 <= 4) return {4, 1};
  if (c8 <= 8) return {4, 2};
  if (c8 <= 12 && !both_backward) return {4, 3};
  if (c8 <= 16) return {8, 2};
  if (c8 <= 24) return {8, 3};
  if (c8 <= 32) return {16, 2};
  if (c8 <= 48) return {16, 3};
  if (c8 <= 64) return {32, 2};
  if (c8 <= 96 && !both_backward) return {32, 3};
  if (c8 <= 128) return {128, 1};
  if (c8 <= 256) return {256, 1};
  if (c8 <= 320 && bf16) return {160, 2};
  if (c8 <= 512) return {256, 2};
  return {512, 2};
}

// Threads of a CTA.
inline int threads_of(const Width &wd, int C) {
  return wd.tpr <= 32 ? block_of(wd.tpr) : ((C >> 3) + 32 * wd.nv - 1) / (32 * wd.nv) * 32;
}

struct Split {
  int64_t chunk;
  int ctas;
};

// Consecutive rows per CTA, as many CTAs as fit on the GPU at once (a wide row's
// CTA with fewer warps than its kernel is bounded for leaves room for more).
inline Split split_rows(int64_t rows, int C, int sms, bool bwd, bool branch, bool pre, bool bf16) {
  const Width wd = width_of(C, bwd && branch && pre, bf16);
  const int threads = threads_of(wd, C), most = block_of(wd.tpr);
  int per_sm = blocks_per_sm(wd.tpr, wd.nv, bwd, branch);
  if (threads < most) {
    const int smem = smem_of(wd.tpr, wd.nv, bwd, branch, pre, bf16 ? 2 : 4);
    // threads an SM: what the kernel is bounded for; the norm's backward takes fewer registers than its bound (88 to 96:
    // 1392 channels 156 -> 138 us)
    const int fit = bwd && !branch && wd.nv == 1 ? 640 : per_sm * most;
    per_sm = std::max(per_sm, std::min(fit / threads, 200 * 1024 / smem));
  }
  const int64_t at_once = wd.tpr > 32 ? 1 : threads / wd.tpr;
  const int64_t groups = (rows + at_once - 1) / at_once;
  const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)sms * per_sm));
  int64_t chunk = (rows + ctas - 1) / ctas;
  chunk = std::max<int64_t>(1, (chunk + at_once - 1) / at_once * at_once);
  return {chunk, (int)((rows + chunk - 1) / chunk)};
}

template <typename T, int TPR, int NV, bool kBwd, bool kBranch, bool kPre>
int launch_one(const RowArgs &a, int ctas, cudaStream_t st) {
  using S = Shape<T, TPR, NV, kBwd, kBranch, kPre>;
  void (*kern)(const RowArgs);
  const int threads = threads_of(width_of(a.C, kBwd && kBranch && kPre, sizeof(T) == 2), a.C);
  // the backward of a CTA's rows is built for all the threads too: with their number from the launch it takes 2 % longer
  // at 1024 channels, 4 % at 2048 and 7 % at 4096 (the forward: no longer)
  constexpr bool kAll = TPR <= 32 || TPR == 160;
  if constexpr (!kBwd) kern = rows_fwd_kernel<T, TPR, kAll, NV, kBranch, kPre>;
  else if constexpr (kAll) kern = rows_bwd_kernel<T, TPR, true, NV, kBranch, kPre>;
  else kern = threads == TPR ? rows_bwd_kernel<T, TPR, true, NV, kBranch, kPre> : rows_bwd_kernel<T, TPR, false, NV, kBranch, kPre>;
  if (S::smem > 40 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem) != cudaSuccess)
    return SWIN_ERR_CUDA;
  kern<<<ctas, threads, S::smem, st>>>(a);
  return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
}

// kBoth: a width that the backward with both norms takes too (width_of).
template <typename T, int TPR, int NV, bool kBoth = true>
int launch_rows(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st) {
  if (bwd) {
    if (branch && pre) {
      if constexpr (kBoth) return launch_one<T, TPR, NV, true, true, true>(a, ctas, st);
      else return SWIN_ERR_UNSUPPORTED;  // not picked
    }
    if (branch) return launch_one<T, TPR, NV, true, true, false>(a, ctas, st);
    return launch_one<T, TPR, NV, true, false, true>(a, ctas, st);
  }
  if (branch && pre) return launch_one<T, TPR, NV, false, true, true>(a, ctas, st);
  if (branch) return launch_one<T, TPR, NV, false, true, false>(a, ctas, st);
  return launch_one<T, TPR, NV, false, false, true>(a, ctas, st);
}

template <typename T>
int launch_width(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st) {
  const Width wd = width_of(a.C, bwd && branch && pre, sizeof(T) == 2);
  if (wd.tpr == 2) return launch_rows<T, 2, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 4 && wd.nv == 1) return launch_rows<T, 4, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 4 && wd.nv == 2) return launch_rows<T, 4, 2>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 4) return launch_rows<T, 4, 3, false>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 8 && wd.nv == 2) return launch_rows<T, 8, 2>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 8) return launch_rows<T, 8, 3>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 16 && wd.nv == 2) return launch_rows<T, 16, 2>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 16) return launch_rows<T, 16, 3>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 32 && wd.nv == 2) return launch_rows<T, 32, 2>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 32) return launch_rows<T, 32, 3, false>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 128) return launch_rows<T, 128, 1>(a, bwd, branch, pre, ctas, st);
  if constexpr (sizeof(T) == 2)
    if (wd.tpr == 160) return launch_rows<T, 160, 2>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 256 && wd.nv == 1) return launch_rows<T, 256, 1>(a, bwd, branch, pre, ctas, st);
  if (wd.tpr == 256) return launch_rows<T, 256, 2>(a, bwd, branch, pre, ctas, st);
  return launch_rows<T, 512, 2>(a, bwd, branch, pre, ctas, st);
}


// One row kernel of either type (swin_rows_bf16.cu, swin_rows_f32.cu).
int launch_bf16(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st);
int launch_f32(const RowArgs &a, bool bwd, bool branch, bool pre, int ctas, cudaStream_t st);

}  // namespace rows
}  // namespace swin
