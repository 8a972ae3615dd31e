// swin_vec8.cuh -- eight channels in registers: loads, stores and arithmetic of
// the kernels that work on rows of channels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace swin {
namespace rows {

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

}  // namespace rows
}  // namespace swin
