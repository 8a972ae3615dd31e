// swin_optim.cu -- the parameters' step: AdamW over many tensors at once, and the
// global norm of their gradients (sm_103a).
//
//   g' = c g, m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2,
//   w = w (1 - lr decay) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Three kernels: sums of squares (with clipping, or for the norm alone), one CTA
// that adds them up and works out the step's factors, and the step. Factors, step
// count and learning rate stay on the device.
//
// What bounds the step: HBM. Every element is 28 bytes with fp32 states (read w,
// g, m, v, write w, m, v), 16 to 18 with states of 8 bits.
// A unit is 256 consecutive elements of a tensor, which is also what one scale of
// an 8-bit state covers: a warp takes a unit at a time, eight elements a lane, and
// finds the largest magnitude by shuffles, so states are rounded in the same pass.
// Tensors come as a table in the kernel's parameters: no copy to the device, and a
// captured call keeps its own.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "swin_calls.cuh"

namespace swin {
namespace {

constexpr int kUnit = 256, kThreads = 256, kWarps = kThreads / 32;
// CTAs an SM. Both kernels live on the loads that their warps have in flight. Norm of
// 317 M fp32 gradients: 3 CTAs 244 us, 4 207, 6 186 (6.8 TB/s, the measured copy rate).
// Step of as many bf16 weights in 8 bits, clipped: 2 1545 us, 3 1310, 4 1139, 5 (which
// spill) 1255.
constexpr int kStepBlocks = 4, kNormBlocks = 6;
constexpr int kMostCtas = 1024;                  // partial sums in the workspace

// ---- the table of tensors ----------------------------------------------------------
enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2, kVector = 4 };  // kVector: eight elements a load
struct Entry {
  void *param;
  float *master;
  const void *grad;
  void *m, *v;
  float *m_scale, *v_scale;
  int64_t n;
  uint32_t unit0;  // its first unit among the table's
  uint32_t flags;
  float decay;
};
struct NormEntry {
  const void *grad;
  int64_t n;
  uint32_t unit0, flags;
};
// A kernel's parameters may take 32 764 bytes; smaller tables launch sooner.
template <typename E, int kCount>
struct Table {
  uint32_t units;
  int count;
  E at[kCount];
};

// The tensor of a unit: the last whose first unit is not behind it.
template <typename TableT>
__device__ __forceinline__ int find(const TableT &t, uint32_t unit) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.at[mid].unit0 <= unit) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// What the step reads from the device.
struct Factors {
  float clip;  // c
  float size;  // lr / (1 - b1^t)
  float root;  // 1 / sqrt(1 - b2^t)
  float lr;
  int go;      // 0: a gradient norm that is not finite
};
constexpr size_t kFactorsBytes = 256;
constexpr size_t kWorkspace = kFactorsBytes + kMostCtas * sizeof(double);

// ---- loads and stores of a lane's eight elements ------------------------------------
// Vector units: elements 8 lane ... 8 lane + 7. Others (a tensor's last, or one that
// starts off its boundary): lane, lane + 32, ...; each warp access is a whole run.
__device__ __forceinline__ void load8(const float *p, float (&f)[8]) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void store8(float *p, const float (&f)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
               "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8]) {
  const uint4 r = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
    w[e] = *reinterpret_cast<const uint32_t *>(&h);
  }
  *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a lane's elements lie in a unit that has `left` of them.
struct Place {
  bool vector;
  int lane, left;
  __device__ __forceinline__ int index(int e) const { return vector ? lane * 8 + e : lane + 32 * e; }
  __device__ __forceinline__ bool has(int e) const { return index(e) < left; }
};

template <typename T>
__device__ __forceinline__ void load(const T *p, const Place &pl, float (&f)[8]) {
  if (pl.vector) {
    load8(p + pl.lane * 8, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = pl.has(e) ? (float)p[pl.index(e)] : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store(T *p, const Place &pl, const float (&f)[8]) {
  if (pl.vector) {
    store8(p + pl.lane * 8, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (pl.has(e)) p[pl.index(e)] = (T)f[e];
  }
}

// ---- states in 8 bits -----------------------------------------------------------------
struct Codes {
  uint32_t w[2];  // e4m3, four to a word
};
__device__ __forceinline__ Codes load_codes(const uint8_t *p, const Place &pl) {
  Codes c = {{0u, 0u}};
  if (pl.vector) {
    const uint2 r = *reinterpret_cast<const uint2 *>(p + pl.lane * 8);
    c.w[0] = r.x;
    c.w[1] = r.y;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (pl.has(e)) c.w[e >> 2] |= (uint32_t)p[pl.index(e)] << (8 * (e & 3));
  }
  return c;
}
__device__ __forceinline__ void store_codes(uint8_t *p, const Place &pl, const Codes &c) {
  if (pl.vector) {
    *reinterpret_cast<uint2 *>(p + pl.lane * 8) = make_uint2(c.w[0], c.w[1]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (pl.has(e)) p[pl.index(e)] = (uint8_t)(c.w[e >> 2] >> (8 * (e & 3)));
  }
}
__device__ __forceinline__ void decode(const Codes &c, float scale, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c.w[e >> 2] >> (8 * (e & 3))), __NV_E4M3);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    f[e] = x.x * scale;
    f[e + 1] = x.y * scale;
  }
}
// Rounds to nearest, times `inverse`. kFloor: what is above 0 is at least the smallest value.
template <bool kFloor>
__device__ __forceinline__ Codes encode(const float (&f)[8], float inverse) {
  Codes c;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w = 0u;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const float2 x = make_float2(f[4 * i + e] * inverse, f[4 * i + e + 1] * inverse);
      uint32_t two = __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3);
      if (kFloor) {
        if (f[4 * i + e] > 0.f && (two & 0xFFu) == 0u) two |= 1u;
        if (f[4 * i + e + 1] > 0.f && (two & 0xFF00u) == 0u) two |= 0x100u;
      }
      w |= two << (8 * e);
    }
    c.w[i] = w;
  }
  return c;
}
__device__ __forceinline__ float largest(const float (&f)[8]) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
  // magnitudes order as their bits do
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
}
// The scale of 256 values whose largest magnitude is `top`, and its inverse (of values that small: zeros).
__device__ __forceinline__ float scale_of(float top, float *inverse) {
  const bool some = top >= 0x1p-100f;
  *inverse = some ? 448.f / top : 0.f;
  return some ? top / 448.f : 0.f;
}

// ---- the step --------------------------------------------------------------------------
struct StepArgs {
  const Factors *factors;
  float beta1, beta2, one1, one2, eps;  // one: 1 - beta
};

// Step of 317 M bf16 weights with fp32 gradients in 8 bits, clipped: 1133 us with the
// norm's 186, so 6.0 TB/s (89 % of the measured copy rate): latency at 32 warps an SM.
// (A form of the loop's body for whole units and each gradient type, so that no
// conversion waits in a branch: 1292 us.)
template <bool k8, int kCount>
__global__ void __launch_bounds__(kThreads, kStepBlocks) step_kernel(const __grid_constant__ Table<Entry, kCount> t,
                                                                     const StepArgs a) {
  const int lane = threadIdx.x & 31;
  // a CTA's units are consecutive, its warps take them in turn
  const uint32_t u0 = (uint32_t)((uint64_t)t.units * blockIdx.x / gridDim.x);
  const uint32_t u1 = (uint32_t)((uint64_t)t.units * (blockIdx.x + 1) / gridDim.x);
  uint32_t u = u0 + (threadIdx.x >> 5);
  int i = u < u1 ? find(t, u) : 0;
  // the factors are there after this; everything else was before the kernel in front
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Factors k = *a.factors;
  if (!k.go) return;
  for (; u < u1; u += kWarps) {
    while (i + 1 < t.count && t.at[i + 1].unit0 <= u) ++i;
    const Entry &en = t.at[i];
    const int64_t at = (int64_t)(u - en.unit0) * kUnit;
    const int left = (int)min((int64_t)kUnit, en.n - at);
    const Place pl = {(en.flags & kVector) && left == kUnit, lane, left};
    float g[8], w[8], m[8], v[8], root[8];
    Codes cm, cv;
    float sm = 0.f, sv = 0.f;
    if (en.flags & kGradBf16) load(static_cast<const __nv_bfloat16 *>(en.grad) + at, pl, g);
    else load(static_cast<const float *>(en.grad) + at, pl, g);
    float *weight = en.flags & kParamBf16 ? en.master : static_cast<float *>(en.param);
    load(weight + at, pl, w);
    if (k8) {
      cm = load_codes(static_cast<const uint8_t *>(en.m) + at, pl);
      cv = load_codes(static_cast<const uint8_t *>(en.v) + at, pl);
      sm = en.m_scale[u - en.unit0];
      sv = en.v_scale[u - en.unit0];
      decode(cm, sm, m);
      decode(cv, sv, v);
    } else {
      load(static_cast<const float *>(en.m) + at, pl, m);
      load(static_cast<const float *>(en.v) + at, pl, v);
    }
    const float keep = 1.f - k.lr * en.decay;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float ge = g[e] * k.clip;
      if (k8) v[e] *= v[e];
      m[e] = fmaf(m[e], a.beta1, ge * a.one1);
      v[e] = fmaf(v[e], a.beta2, ge * ge * a.one2);
      root[e] = sqrtf(v[e]);
      w[e] = fmaf(w[e], keep, -k.size * m[e] / fmaf(root[e], k.root, a.eps));
    }
    store(weight + at, pl, w);
    if (en.flags & kParamBf16) store(static_cast<__nv_bfloat16 *>(en.param) + at, pl, w);
    if (k8) {
      float im, iv;
      sm = scale_of(largest(m), &im);
      sv = scale_of(largest(root), &iv);
      store_codes(static_cast<uint8_t *>(en.m) + at, pl, encode<false>(m, im));
      store_codes(static_cast<uint8_t *>(en.v) + at, pl, encode<true>(root, iv));
      if (lane == 0) {
        en.m_scale[u - en.unit0] = sm;
        en.v_scale[u - en.unit0] = sv;
      }
    } else {
      store(static_cast<float *>(en.m) + at, pl, m);
      store(static_cast<float *>(en.v) + at, pl, v);
    }
  }
}

// ---- the norm ---------------------------------------------------------------------------
// Squares are fp32; sixteen units' worth of a lane's are added in fp32 (16 deep, in eight
// sums of their own), then in fp64.
template <int kCount>
__global__ void __launch_bounds__(kThreads, kNormBlocks) squares_kernel(const __grid_constant__ Table<NormEntry, kCount> t,
                                                                        double *sums) {
  const int lane = threadIdx.x & 31;
  const uint32_t u0 = (uint32_t)((uint64_t)t.units * blockIdx.x / gridDim.x);
  const uint32_t u1 = (uint32_t)((uint64_t)t.units * (blockIdx.x + 1) / gridDim.x);
  uint32_t u = u0 + (threadIdx.x >> 5);
  int i = u < u1 ? find(t, u) : 0;
  double all = 0.0;
  while (u < u1) {
    float s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = 0.f;
#pragma unroll 4
    for (int r = 0; r < 16 && u < u1; ++r, u += kWarps) {
      while (i + 1 < t.count && t.at[i + 1].unit0 <= u) ++i;
      const NormEntry &en = t.at[i];
      const int64_t at = (int64_t)(u - en.unit0) * kUnit;
      const int left = (int)min((int64_t)kUnit, en.n - at);
      const Place pl = {(en.flags & kVector) && left == kUnit, lane, left};
      float g[8];
      if (en.flags & kGradBf16) load(static_cast<const __nv_bfloat16 *>(en.grad) + at, pl, g);
      else load(static_cast<const float *>(en.grad) + at, pl, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[e] = fmaf(g[e], g[e], s[e]);
    }
    all += (double)(((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7])));
  }
  __shared__ double buf[kWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
  if (lane == 0) buf[threadIdx.x >> 5] = all;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int w = 1; w < kWarps; ++w) all += buf[w];
    sums[blockIdx.x] = all;
  }
}

struct FinishArgs {
  const double *sums;
  int count;        // of sums
  float *norm;      // or NULL
  Factors *factors; // NULL: the norm alone
  const float *lr;
  int64_t *steps;
  double beta1, beta2, max_norm;
};

__global__ void __launch_bounds__(kThreads) finish_kernel(const FinishArgs a) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ double buf[kWarps];
  double s = 0.0;
  for (int i = threadIdx.x; i < a.count; i += kThreads) s += a.sums[i];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) s += buf[w];
  const double norm = sqrt(s);
  if (a.norm) *a.norm = (float)norm;
  if (!a.factors) return;
  const int64_t steps = *a.steps + 1;
  Factors f;
  f.go = isfinite((float)norm);
  f.clip = a.count && norm > a.max_norm ? (float)(a.max_norm / norm) : 1.f;
  f.lr = *a.lr;
  f.size = (float)((double)f.lr / (1.0 - pow(a.beta1, (double)steps)));
  f.root = (float)(1.0 / sqrt(1.0 - pow(a.beta2, (double)steps)));
  *a.factors = f;
  if (f.go) *a.steps = steps;
}

// ---- host --------------------------------------------------------------------------------
bool of_type(int32_t t) { return t == SWIN_F32 || t == SWIN_BF16; }
int64_t size_of(int32_t t) { return t == SWIN_BF16 ? 2 : 4; }
uint32_t units_of(int64_t n) { return (uint32_t)((n + kUnit - 1) / kUnit); }

bool taken(const swin_attn_param &p) { return p.n > 0 && p.grad; }

int check_gradients(const swin_attn_param *p, int64_t count) {
  if (count < 0 || (count && !p)) return SWIN_ERR_INVALID_ARG;
  int64_t all = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (p[i].n < 0) return SWIN_ERR_INVALID_ARG;
    if (!of_type(p[i].grad_dtype)) return SWIN_ERR_UNSUPPORTED;
    if (!taken(p[i])) continue;
    if (p[i].n >= (int64_t(1) << 39) || (all += (p[i].n + kUnit - 1) / kUnit * kUnit) >= (int64_t(1) << 39))
      return SWIN_ERR_UNSUPPORTED;
    if (mis(p[i].grad, size_of(p[i].grad_dtype))) return SWIN_ERR_ALIGNMENT;
  }
  return SWIN_OK;
}

struct Range {
  uintptr_t begin, end;
  bool operator<(const Range &o) const { return begin < o.begin; }
};
Range range(const void *p, int64_t bytes) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(p);
  return {b, b + (uintptr_t)bytes};
}
// Outputs that overlap one another, or an input.
bool clash(std::vector<Range> &out, const std::vector<Range> &in) {
  std::sort(out.begin(), out.end());
  for (size_t i = 1; i < out.size(); ++i)
    if (out[i].begin < out[i - 1].end) return true;
  for (const Range &r : in) {
    auto next = std::lower_bound(out.begin(), out.end(), r);  // the first that begins at or behind r
    if (next != out.end() && next->begin < r.end) return true;
    if (next != out.begin() && (next - 1)->end > r.begin) return true;
  }
  return false;
}

Entry entry_of(const swin_attn_param &p, bool k8) {
  Entry e = {p.param, p.master, p.grad, p.m, p.v, p.m_scale, p.v_scale, p.n, 0u, 0u, p.decay};
  const bool half = p.dtype == SWIN_BF16, grad_half = p.grad_dtype == SWIN_BF16;
  e.flags = (half ? kParamBf16 : 0u) | (grad_half ? kGradBf16 : 0u);
  const int state = k8 ? 8 : 32;
  if (!mis(p.param, half ? 16 : 32) && !mis(p.master, 32) && !mis(p.grad, grad_half ? 16 : 32) && !mis(p.m, state) &&
      !mis(p.v, state))
    e.flags |= kVector;
  return e;
}
NormEntry norm_entry_of(const swin_attn_param &p) {
  const bool half = p.grad_dtype == SWIN_BF16;
  return {p.grad, p.n, 0u, (half ? kGradBf16 : 0u) | (mis(p.grad, half ? 16 : 32) ? 0u : kVector)};
}

// Calls launch(table) for the next taken tensors, as many as a table holds. (Their units are below 2^31.)
template <int kCount, typename E, typename Make, typename Launch>
int table_of(const swin_attn_param *p, int64_t count, int64_t &next, Make make, Launch launch) {
  Table<E, kCount> t;
  t.units = 0;
  t.count = 0;
  for (; next < count && t.count < kCount; ++next) {
    if (!taken(p[next])) continue;
    E e = make(p[next]);
    e.unit0 = t.units;
    t.at[t.count++] = e;
    t.units += units_of(p[next].n);
  }
  if (!t.count) return SWIN_OK;
  if (t.count < kCount) std::memset(static_cast<void *>(&t.at[t.count]), 0, sizeof(E) * (kCount - t.count));
  return launch(t);
}

int ctas_of(uint32_t units, int most) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(most, ((int64_t)units + kWarps - 1) / kWarps));
}

constexpr int kSmall = 24, kLarge = 400;  // step tables: 1.9 and 31 KB
constexpr int kNormSmall = 64, kNormLarge = 1024;

int64_t taken_of(const swin_attn_param *p, int64_t count) {
  int64_t some = 0;
  for (int64_t i = 0; i < count; ++i) some += taken(p[i]);
  return some;
}

// Sums of squares of all gradients; *slots: how many.
int launch_squares(const swin_attn_param *p, int64_t count, double *sums, int *slots, int sms, cudaStream_t st) {
  const int64_t some = taken_of(p, count), rounds = (some + kNormLarge - 1) / kNormLarge;
  *slots = 0;
  if (rounds > kMostCtas) return SWIN_ERR_UNSUPPORTED;
  const int most = std::min<int>(sms * kNormBlocks, rounds ? (int)(kMostCtas / rounds) : kMostCtas);
  auto launch = [&](const auto &t) {
    const int ctas = ctas_of(t.units, most);
    squares_kernel<<<ctas, kThreads, 0, st>>>(t, sums + *slots);
    *slots += ctas;
    return cudaPeekAtLastError() == cudaSuccess ? SWIN_OK : SWIN_ERR_CUDA;
  };
  for (int64_t next = 0; next < count;) {
    const int rc = some <= kNormSmall ? table_of<kNormSmall, NormEntry>(p, count, next, norm_entry_of, launch)
                                      : table_of<kNormLarge, NormEntry>(p, count, next, norm_entry_of, launch);
    if (rc) return rc;
  }
  return SWIN_OK;
}

template <bool k8>
int launch_steps(const swin_attn_param *p, int64_t count, const StepArgs &a, int sms, cudaStream_t st) {
  const int64_t some = taken_of(p, count);
  auto make = [](const swin_attn_param &q) { return entry_of(q, k8); };
  const dim3 block(kThreads);
  auto small = [&](const Table<Entry, kSmall> &t) {
    return launch_dependent(step_kernel<k8, kSmall>, dim3(ctas_of(t.units, sms * kStepBlocks)), block, 0, st, t, a);
  };
  auto large = [&](const Table<Entry, kLarge> &t) {
    return launch_dependent(step_kernel<k8, kLarge>, dim3(ctas_of(t.units, sms * kStepBlocks)), block, 0, st, t, a);
  };
  for (int64_t next = 0; next < count;) {
    const int rc = some <= kSmall ? table_of<kSmall, Entry>(p, count, next, make, small)
                                  : table_of<kLarge, Entry>(p, count, next, make, large);
    if (rc) return rc;
  }
  return SWIN_OK;
}

}  // namespace
}  // namespace swin

using namespace swin;

extern "C" {

size_t swin_attn_adamw_workspace_bytes(void) { return kWorkspace; }

int swin_attn_grad_norm(const swin_attn_param *params, int64_t count, float *norm, void *workspace,
                        size_t workspace_bytes, swin_stream_t stream) {
  int rc = check_gradients(params, count);
  if (rc) return rc;
  if (!norm) return SWIN_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < kWorkspace) return SWIN_ERR_WORKSPACE;
  if (mis(norm, 4) || mis(workspace, 256)) return SWIN_ERR_ALIGNMENT;
  std::vector<Range> out = {range(norm, 4), range(workspace, kWorkspace)}, in;
  for (int64_t i = 0; i < count; ++i)
    if (taken(params[i])) in.push_back(range(params[i].grad, params[i].n * size_of(params[i].grad_dtype)));
  if (clash(out, in)) return SWIN_ERR_INVALID_ARG;
  int sms = 0, slots = 0;
  if ((rc = sm_count(&sms))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  double *sums = reinterpret_cast<double *>(static_cast<uint8_t *>(workspace) + kFactorsBytes);
  if ((rc = launch_squares(params, count, sums, &slots, sms, st))) return rc;
  FinishArgs f = {};
  f.sums = sums;
  f.count = slots;
  f.norm = norm;
  return launch_dependent(finish_kernel, dim3(1), dim3(kThreads), 0, st, f);
}

int swin_attn_adamw_step(const swin_attn_adamw *o, const swin_attn_param *params, int64_t count, void *workspace,
                         size_t workspace_bytes, swin_stream_t stream) {
  int rc = check_gradients(params, count);
  if (rc) return rc;
  if (!o || !o->lr || !o->steps) return SWIN_ERR_INVALID_ARG;
  if (!(o->beta1 >= 0.0 && o->beta1 < 1.0) || !(o->beta2 >= 0.0 && o->beta2 < 1.0)) return SWIN_ERR_INVALID_ARG;
  if (!(o->eps > 0.0) || !std::isfinite((float)o->eps) || !((float)o->eps > 0.f)) return SWIN_ERR_INVALID_ARG;
  if (!(o->max_norm >= 0.0) || !std::isfinite(o->max_norm)) return SWIN_ERR_INVALID_ARG;
  if (o->norm && o->max_norm == 0.0) return SWIN_ERR_INVALID_ARG;
  if (o->state_bits != 32 && o->state_bits != 8) return SWIN_ERR_UNSUPPORTED;
  if (mis(o->lr, 4) || mis(o->steps, 8) || mis(o->norm, 4)) return SWIN_ERR_ALIGNMENT;
  const bool k8 = o->state_bits == 8;
  std::vector<Range> out, in;
  out.reserve(6 * (size_t)count + 3);
  in.reserve((size_t)count + 1);
  for (int64_t i = 0; i < count; ++i) {
    const swin_attn_param &p = params[i];
    if (!of_type(p.dtype)) return SWIN_ERR_UNSUPPORTED;
    if (!(p.decay >= 0.f) || !std::isfinite(p.decay)) return SWIN_ERR_INVALID_ARG;
    if (!taken(p)) continue;
    if (!p.param || !p.m || !p.v || (p.dtype == SWIN_BF16) != (p.master != nullptr) ||
        k8 != (p.m_scale != nullptr) || k8 != (p.v_scale != nullptr))
      return SWIN_ERR_INVALID_ARG;
    if (mis(p.param, size_of(p.dtype)) || mis(p.master, 4) || mis(p.m_scale, 4) || mis(p.v_scale, 4) ||
        (!k8 && (mis(p.m, 4) || mis(p.v, 4))))
      return SWIN_ERR_ALIGNMENT;
    const int64_t scales = (int64_t)units_of(p.n) * 4;
    out.push_back(range(p.param, p.n * size_of(p.dtype)));
    if (p.master) out.push_back(range(p.master, p.n * 4));
    out.push_back(range(p.m, p.n * (k8 ? 1 : 4)));
    out.push_back(range(p.v, p.n * (k8 ? 1 : 4)));
    if (k8) {
      out.push_back(range(p.m_scale, scales));
      out.push_back(range(p.v_scale, scales));
    }
    in.push_back(range(p.grad, p.n * size_of(p.grad_dtype)));
  }
  if (!workspace || workspace_bytes < kWorkspace) return SWIN_ERR_WORKSPACE;
  if (mis(workspace, 256)) return SWIN_ERR_ALIGNMENT;
  out.push_back(range(workspace, kWorkspace));
  out.push_back(range(o->steps, 8));
  if (o->norm) out.push_back(range(o->norm, 4));
  in.push_back(range(o->lr, 4));
  if (clash(out, in)) return SWIN_ERR_INVALID_ARG;
  int sms = 0, slots = 0;
  if ((rc = sm_count(&sms))) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  Factors *factors = static_cast<Factors *>(workspace);
  double *sums = reinterpret_cast<double *>(static_cast<uint8_t *>(workspace) + kFactorsBytes);
  if (o->max_norm > 0.0 && (rc = launch_squares(params, count, sums, &slots, sms, st))) return rc;
  FinishArgs f = {};
  f.sums = sums;
  f.count = slots;
  f.norm = o->norm;
  f.factors = factors;
  f.lr = o->lr;
  f.steps = o->steps;
  f.beta1 = o->beta1;
  f.beta2 = o->beta2;
  f.max_norm = o->max_norm;
  if (slots) {
    if ((rc = launch_dependent(finish_kernel, dim3(1), dim3(kThreads), 0, st, f))) return rc;
  } else {  // the first kernel of the call: what came before it is done when it starts
    finish_kernel<<<1, kThreads, 0, st>>>(f);
    if (cudaPeekAtLastError() != cudaSuccess) return SWIN_ERR_CUDA;
  }
  const StepArgs a = {factors, (float)o->beta1, (float)o->beta2, (float)(1.0 - o->beta1), (float)(1.0 - o->beta2),
                      (float)o->eps};
  return k8 ? launch_steps<true>(params, count, a, sms, st) : launch_steps<false>(params, count, a, sms, st);
}

}  // extern "C"
