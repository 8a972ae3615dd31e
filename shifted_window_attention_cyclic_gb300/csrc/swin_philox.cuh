// swin_philox.cuh -- dropout decisions from a counter-based generator.
//
// Philox4x32-7 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011; seven rounds are the fewest the paper reports to pass
// every BigCrush test): the 64-bit seed is the key, the counter is (block low,
// block high, site, step). One block's 128 bits are eight 16-bit numbers, so
// eight decisions: decision i is number i % 8 of block i / 8 (word (i % 8) / 2,
// low half first) and keeps iff the number is >= T = rint(rate * 65536). A
// decision is a pure function of (seed, step, site, i): forward and backward
// recompute it, whatever tiles their kernels use, and no mask is stored.
// 16 bits per decision, not 32: half the generator's work, and rates are
// honoured to 2^-17; the kept values' scale is 1 / (1 - T / 65536), the exact
// inverse of the share that is kept.
#pragma once
#include <cmath>
#include <cstdint>

#include "../../include/swin_attn.h"

namespace swin {

// A dropout as the kernels take it; thr == 0 means none.
struct Drop {
  uint32_t thr;           // T
  uint32_t site;
  float scale;            // 65536 / (65536 - T)
  const uint64_t *state;  // device: {seed, step}
};

// Checks and converts the caller's descriptor (NULL or rate 0: no dropout).
inline int make_drop(const swin_attn_drop *d, Drop *out) {
  *out = Drop{0u, 0u, 1.f, nullptr};
  if (!d) return SWIN_OK;
  if (!(d->rate >= 0.0 && d->rate < 1.0)) return SWIN_ERR_INVALID_ARG;
  const double t = std::rint(d->rate * 65536.0);
  if (t == 0.0) return SWIN_OK;
  if (t > 65535.0 || !d->state) return SWIN_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(d->state) & 7u) return SWIN_ERR_ALIGNMENT;
  out->thr = (uint32_t)t;
  out->site = d->site;
  out->scale = (float)(65536.0 / (65536.0 - t));
  out->state = d->state;
  return SWIN_OK;
}

// The generator of one dropout in one launch.
struct Philox {
  uint32_t k0, k1, site, step;

  __device__ __forceinline__ void init(const Drop &d) {
    k0 = k1 = step = 0u;
    site = d.site;
    if (d.thr) {
      const uint64_t seed = __ldg(reinterpret_cast<const unsigned long long *>(d.state));
      k0 = (uint32_t)seed;
      k1 = (uint32_t)(seed >> 32);
      step = (uint32_t)__ldg(reinterpret_cast<const unsigned long long *>(d.state) + 1);
    }
  }

  // The eight 16-bit numbers of a block, two per word, low half first.
  __device__ __forceinline__ uint4 block(uint64_t b) const {
    uint32_t c0 = (uint32_t)b, c1 = (uint32_t)(b >> 32), c2 = site, c3 = step, a = k0, k = k1;
#pragma unroll
    for (int r = 0; r < 7; ++r) {
      const uint64_t p0 = (uint64_t)c0 * 0xD2511F53u, p1 = (uint64_t)c2 * 0xCD9E8D57u;
      c0 = (uint32_t)(p1 >> 32) ^ c1 ^ a;
      c1 = (uint32_t)p1;
      c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k;
      c3 = (uint32_t)p0;
      a += 0x9E3779B9u;
      k += 0xBB67AE85u;
    }
    return make_uint4(c0, c1, c2, c3);
  }

  // N blocks, a round of all at a time: independent chains (a wide multiply
  // issues every fourth cycle at best, and a lone chain waits for each).
  template <int N>
  __device__ __forceinline__ void blocks(const uint64_t (&b)[N], uint4 (&u)[N]) const {
    uint32_t a = k0, k = k1;
#pragma unroll
    for (int i = 0; i < N; ++i) u[i] = make_uint4((uint32_t)b[i], (uint32_t)(b[i] >> 32), site, step);
#pragma unroll
    for (int r = 0; r < 7; ++r) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint64_t p0 = (uint64_t)u[i].x * 0xD2511F53u, p1 = (uint64_t)u[i].z * 0xCD9E8D57u;
        u[i] = make_uint4((uint32_t)(p1 >> 32) ^ u[i].y ^ a, (uint32_t)p1, (uint32_t)(p0 >> 32) ^ u[i].w ^ k, (uint32_t)p0);
      }
      a += 0x9E3779B9u;
      k += 0xBB67AE85u;
    }
  }
};

// Decision e (a compile-time 0..7 after unrolling) of a block. The number is
// compared in a word's upper half, where T << 16 sits: the odd ones as they
// are (their lower half cannot change the outcome), the even ones moved up.
__device__ __forceinline__ bool keep_of(const uint4 &u, int e, uint32_t thr) {
  const uint32_t w = e < 2 ? u.x : e < 4 ? u.y : e < 6 ? u.z : u.w;
  return ((e & 1) ? w : w << 16) >= thr << 16;
}

// Both decisions of a generator word at once, as the sign bits of its halves
// (the other bits are not defined): with 15-bit values, u + (0x8000 - T) carries
// into bit 15 iff u >= T. For T <= 0x8000 a number with its own top bit set
// keeps whatever the rest; above, only such a number can keep.
struct PairTest {
  uint32_t add, any;
  __device__ __forceinline__ void init(uint32_t thr) {
    any = thr <= 0x8000u ? ~0u : 0u;
    add = (0x8000u - (thr <= 0x8000u ? thr : thr - 0x8000u)) * 0x10001u;
  }
  __device__ __forceinline__ uint32_t signs(uint32_t w) const {
    const uint32_t t = (w & 0x7FFF7FFFu) + add;
    return (t & w) | (any & (t | w));
  }
};

// The decisions of a 16-key group (two generator blocks) as four bits in each
// byte: key 4 k + j at bit k of byte j. The signs of four halves become four
// bytes of ones or zeros in one byte permute (selectors that replicate a sign),
// so two words cost one permute and one LOP.
__device__ __forceinline__ uint32_t group_bits(const uint4 &a, const uint4 &b, const PairTest &test) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t bits = 0u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t m;
    asm("prmt.b32 %0, %1, %2, 0xFDB9;" : "=r"(m) : "r"(test.signs(w[2 * k])), "r"(test.signs(w[2 * k + 1])));
    bits |= m & (0x01010101u << k);
  }
  return bits;
}
// 0xFFFF in the halves that keep, 0 in the others, of keys e and e + 1 (e even) of a group.
__device__ __forceinline__ uint32_t keep_mask(uint32_t bits, int e) {
  uint32_t m;
  if (e & 2)
    asm("prmt.b32 %0, %1, 0, 0xBBAA;" : "=r"(m) : "r"(bits << (7 - (e >> 2))));
  else
    asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(m) : "r"(bits << (7 - (e >> 2))));
  return m;
}
// Key e of a group alone.
__device__ __forceinline__ bool keep_bit(uint32_t bits, int e) { return (bits & (1u << (8 * (e & 3) + (e >> 2)))) != 0u; }

// The decisions of attention probabilities: row (image b, head h, query token t),
// key slots in order, ceil(n / 8) blocks a row.
struct KeepDraw {
  Philox ph;
  PairTest test;
  int nb;
  __device__ __forceinline__ void init(const Drop &d, int n) {
    ph.init(d);
    test.init(d.thr);
    nb = (n + 7) >> 3;
  }
  // first block of a query's row (a pad, token -1: any row will do)
  __device__ __forceinline__ uint64_t row(int b, int h, int heads, int tokens, int token) const {
    return (((uint64_t)b * heads + h) * tokens + max(token, 0)) * nb;
  }
  // the 16-key group whose first block is b (group_bits)
  __device__ __forceinline__ uint32_t group(uint64_t b) const {
    const uint64_t at[2] = {b, b + 1};
    uint4 r[2];
    ph.blocks(at, r);
    return group_bits(r[0], r[1], test);
  }
};

// A block's eight decisions, bit e = decision e keeps.
__device__ __forceinline__ uint32_t keep_bits(const uint4 &u, uint32_t thr) {
  uint32_t m = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) m |= keep_of(u, e, thr) ? 1u << e : 0u;
  return m;
}

// One decision, alone.
__device__ __forceinline__ bool keep_one(const Philox &ph, uint64_t i, uint32_t thr) {
  const uint4 u = ph.block(i >> 3);
  const int e = (int)(i & 7);
  const uint32_t w = (e >> 1) == 0 ? u.x : (e >> 1) == 1 ? u.y : (e >> 1) == 2 ? u.z : u.w;
  return ((e & 1) ? (w >> 16) : (w & 0xFFFFu)) >= thr;
}

}  // namespace swin
