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
#include <atomic>
#include <cmath>

#include "swin_rows.cuh"

namespace swin {
namespace {

using namespace rows;

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
// cold caches, 3 to 6 us behind the row kernel, whose sums lie in L2. (Blocks of 8
// channels and 128 lanes: join backward of 256 channels 1 to 2 us shorter, of
// 4096 channels 8 longer; of 16 channels: 0 and 4. Eight slots loaded at once
// under predicates: 2 us longer with 1024 channels, else the same.)
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
    // every parameter is read before a gradient is written: each may lie on its parameter
    const float scale = at(a.scale, c, 1.f), g = at(gamma, c, 1.f), b = at(beta, c, 0.f);
    if (a.dpost_gamma) a.dpost_gamma[c] = a.kept * scale * all.one;
    if (a.dpost_beta) a.dpost_beta[c] = a.kept * scale * all.zero;
    if (a.dscale) a.dscale[c] = a.kept * fmaf(g, all.one, b * all.zero);
  }
}

// ---- dropout -------------------------------------------------------------------
// Element i keeps iff decision i / span does. kMode 0: span 1, one block per
// 8-element vector; 1: span a multiple of 8, one decision per vector; 2: any
// other span, whose vectors need up to eight decisions of at most two blocks.
// 302 M bf16 elements, span 1: 187 us, 6.4 TB/s (95 % of the measured copy rate):
// HBM; the generator's wide multiplies fill 57 % of their pipe.
template <typename T, int kMode>
__global__ void __launch_bounds__(256) dropout_kernel(const T *x, T *y, int64_t n, int64_t span, Drop d, bool wide) {
  Philox ph;
  ph.init(d);
  const int64_t nvec = (n + 7) >> 3;
  const bool narrow = n <= UINT32_MAX;  // 32-bit division: a quarter of the long one's work
  for (int64_t v = (int64_t)blockIdx.x * 256 + threadIdx.x; v < nvec; v += (int64_t)gridDim.x * 256) {
    const int64_t i0 = v * 8;
    uint4 own = make_uint4(0u, 0u, 0u, 0u);  // modes 0 and 1: numbers compared where they are used (as bits: 201 us)
    uint32_t keep = 0u;                      // mode 2, bit e: element i0 + e keeps
    if (kMode == 0) {
      own = ph.block((uint64_t)v);
    } else {
      const int64_t first = narrow ? (uint32_t)i0 / (uint32_t)min(span, (int64_t)UINT32_MAX) : i0 / span;
      if (kMode == 1) {
        if (keep_one(ph, (uint64_t)first, d.thr)) own = make_uint4(~0u, ~0u, ~0u, ~0u);
      } else {
        const uint64_t at[2] = {(uint64_t)first >> 3, ((uint64_t)first >> 3) + 1};
        uint4 r[2];
        ph.blocks(at, r);
        uint32_t bits = (keep_bits(r[0], d.thr) | keep_bits(r[1], d.thr) << 8) >> (first & 7);
        int64_t left = span - (i0 - first * span);  // elements of the decision still to come
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          keep |= (bits & 1u) << e;
          if (--left == 0) {
            left = span;
            bits >>= 1;
          }
        }
      }
    }
    if (i0 + 8 <= n) {
      Raw<T> in;
      load8(x + i0, in, wide);
      float2 f[4];
      unpack(in, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        f[e] = mul(f[e], both(d.scale));
        if (kMode < 2) f[e] = kept(own, e, d.thr, f[e]);
        else f[e] = make_float2((keep >> (2 * e)) & 1u ? f[e].x : 0.f, (keep >> (2 * e + 1)) & 1u ? f[e].y : 0.f);
      }
      Raw<T> out;
      pack(f, out);
      store8(y, i0 * (int64_t)sizeof(T), out, wide);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i0 + e < n) {
          const bool k = kMode < 2 ? keep_of(own, e, d.thr) : (keep >> e) & 1u;
          y[i0 + e] = (T)(k ? (float)x[i0 + e] * d.scale : 0.f);
        }
    }
  }
}

// ---- launches ----------------------------------------------------------------------
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

// What a call reads or writes. An output may lie exactly on an input of its own
// kind and size: an activation on an activation (each is read before its place
// is written, by the same thread or warp), a parameter's gradient on that
// parameter (the fold writes when nothing reads it any more). Any other overlap
// would be a race.
enum Kind { kActivation, kPostGamma, kPostBeta, kScale, kGate, kPreGamma, kPreBeta, kState, kWorkspace };
struct Range {
  const void *at;
  size_t bytes;
  Kind kind;
};
bool meet(const Range &a, const Range &b) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
  return p && q && a.bytes && b.bytes && p < q + b.bytes && q < p + a.bytes;
}
template <int kOut, int kIn>
bool clash(const Range (&out)[kOut], const Range (&in)[kIn]) {
  for (int i = 0; i < kOut; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return true;
    for (const Range &r : in)
      if (meet(out[i], r) && !(r.kind == out[i].kind && r.at == out[i].at && r.bytes == out[i].bytes)) return true;
  }
  return false;
}
Range state_of(const Drop &d) { return {d.state, 2 * sizeof(uint64_t), kState}; }

// Column sums in the workspace: of the pre norm [ctas], of the join [ctas + images with rows], of image groups.
int64_t join_slots(int ctas, int64_t images, int64_t rows) {
  return (int64_t)ctas + std::max<int64_t>(std::min(images, rows), 1);
}
int64_t image_groups(int64_t images) { return std::max<int64_t>(1, (images + kGroupImages - 1) / kGroupImages); }

// Bytes of a backward's workspace, whichever of its kernels runs; images: 1 where there is no gate.
size_t workspace_bytes_of(const swin_attn_rows *r, int64_t images, int sms) {
  const int64_t rows = r->images * r->tokens;
  int ctas = 0;
  for (int k = 1; k < 4; ++k)
    ctas = std::max(ctas, split_rows(rows, r->channels, sms, true, k & 1, k & 2, r->dtype == SWIN_BF16).ctas);
  const size_t slots = (size_t)(ctas + join_slots(ctas, images, rows) + image_groups(images));
  const size_t need = slots * 2 * r->channels * sizeof(float);
  return (need + 255) & ~size_t(255);
}

// The images that a join's rows are cut by: where neither gate nor path looks at
// them, one (every image a CTA meets costs it a drained and refilled ring).
void cut_images(const swin_attn_rows *r, RowArgs *a) {
  const bool any = a->gate || a->path.thr;
  a->tokens = any ? r->tokens : a->rows;
  a->images = any ? (int)r->images : 1;
}

}  // namespace
}  // namespace swin

using namespace swin;

extern "C" {

size_t swin_attn_rows_workspace_bytes(const swin_attn_rows *r) {
  int64_t rows = 0;
  size_t bytes = 0;
  int sms = 0;
  if (check_rows(r, &rows, &bytes) || sm_count(&sms)) return 0;
  return workspace_bytes_of(r, r->images, sms);
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
  if (!x || !h) return SWIN_ERR_INVALID_ARG;
  const size_t cb = sizeof(float) * r->channels;
  const Range out[] = {{h, bytes, kActivation}};
  const Range in[] = {{x, bytes, kActivation}, {norm->gamma, cb, kPreGamma}, {norm->beta, cb, kPreBeta}};
  if (clash(out, in)) return SWIN_ERR_INVALID_ARG;
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
  const Split sp = split_rows(a.rows, a.C, sms, false, false, true, r->dtype == SWIN_BF16);
  a.chunk = sp.chunk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return r->dtype == SWIN_BF16 ? launch_bf16(a, false, false, true, sp.ctas, st)
                               : launch_f32(a, false, false, true, sp.ctas, st);
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
  const size_t cb = sizeof(float) * r->channels;
  const Range out[] = {{y, bytes, kActivation}, {h, bytes, kActivation}};
  const Range in[] = {{x, bytes, kActivation},
                      {z, bytes, kActivation},
                      {join->post.gamma, cb, kPostGamma},
                      {join->post.beta, cb, kPostBeta},
                      {join->scale, cb, kScale},
                      {join->gate, cb * r->images, kGate},
                      {join->pre.gamma, cb, kPreGamma},
                      {join->pre.beta, cb, kPreBeta},
                      state_of(a.drop),
                      state_of(a.path)};
  if (clash(out, in)) return SWIN_ERR_INVALID_ARG;
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
  cut_images(r, &a);
  a.C = r->channels;
  const Split sp = split_rows(a.rows, a.C, sms, false, true, pre, r->dtype == SWIN_BF16);
  a.chunk = sp.chunk;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return r->dtype == SWIN_BF16 ? launch_bf16(a, false, true, pre, sp.ctas, st)
                               : launch_f32(a, false, true, pre, sp.ctas, st);
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
  cut_images(r, &a);
  const int64_t groups = a.gate && want_post ? image_groups(a.images) : 1;
  if (groups > 65535) return SWIN_ERR_UNSUPPORTED;  // (a grid's y)
  const Split sp = split_rows(a.rows, a.C, sms, true, branch, pre, r->dtype == SWIN_BF16);
  a.chunk = sp.chunk;
  if (want_pre || want_post) {
    if (!workspace || workspace_bytes < workspace_bytes_of(r, a.gate ? a.images : 1, sms)) return SWIN_ERR_WORKSPACE;
    if (mis(workspace, 256)) return SWIN_ERR_ALIGNMENT;
    float *ws = static_cast<float *>(workspace);
    a.part_pre = want_pre ? ws : nullptr;
    a.part_post = want_post ? ws + (size_t)sp.ctas * 2 * a.C : nullptr;
  }
  if (!pre) {  // of a join whose h no gradient reached
    const size_t cb = sizeof(float) * a.C;
    if (g.pre_gamma && cudaMemsetAsync(g.pre_gamma, 0, cb, st) != cudaSuccess) return SWIN_ERR_CUDA;
    if (g.pre_beta && cudaMemsetAsync(g.pre_beta, 0, cb, st) != cudaSuccess) return SWIN_ERR_CUDA;
  }
  if (a.rows) {
    rc = r->dtype == SWIN_BF16 ? launch_bf16(a, true, branch, pre, sp.ctas, st)
                               : launch_f32(a, true, branch, pre, sp.ctas, st);
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
  if (groups > 1) c.groups = a.part_post + join_slots(sp.ctas, a.images, a.rows) * 2 * a.C;
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
  if (a.rows && (!x || !dh || !dx)) return SWIN_ERR_INVALID_ARG;
  const size_t cb = sizeof(float) * r->channels;
  const Range out[] = {{dx, bytes, kActivation},
                       {dgamma, cb, kPreGamma},
                       {dbeta, cb, kPreBeta},
                       {dgamma || dbeta ? workspace : nullptr, workspace_bytes, kWorkspace}};
  const Range in[] = {{x, bytes, kActivation},
                      {dh, bytes, kActivation},
                      {dres, bytes, kActivation},
                      {norm->gamma, cb, kPreGamma},
                      {norm->beta, cb, kPreBeta}};
  if (clash(out, in)) return SWIN_ERR_INVALID_ARG;
  if (a.rows) {
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
  }
  const size_t cb = sizeof(float) * r->channels, gb = cb * r->images;
  const bool want = grads->post_gamma || grads->post_beta || grads->scale || grads->gate || grads->pre_gamma ||
                    grads->pre_beta;
  const Range out[] = {{dx, bytes, kActivation},
                       {dz, bytes, kActivation},
                       {grads->post_gamma, cb, kPostGamma},
                       {grads->post_beta, cb, kPostBeta},
                       {grads->scale, cb, kScale},
                       {grads->gate, gb, kGate},
                       {grads->pre_gamma, cb, kPreGamma},
                       {grads->pre_beta, cb, kPreBeta},
                       {want ? workspace : nullptr, workspace_bytes, kWorkspace}};
  const Range in[] = {{y, bytes, kActivation},
                      {z, bytes, kActivation},
                      {dy, bytes, kActivation},
                      {dh, bytes, kActivation},
                      {join->post.gamma, cb, kPostGamma},
                      {join->post.beta, cb, kPostBeta},
                      {join->scale, cb, kScale},
                      {join->gate, gb, kGate},
                      {join->pre.gamma, cb, kPreGamma},
                      {join->pre.beta, cb, kPreBeta},
                      state_of(a.drop),
                      state_of(a.path)};
  if (clash(out, in)) return SWIN_ERR_INVALID_ARG;
  if (a.rows) {
    const void *act[6] = {y, z, dy, dh, dx, dz};
    for (const void *p : act)
      if (mis(p, 16)) return SWIN_ERR_ALIGNMENT;
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
  return run_backward(a, r, true, *grads, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
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
  if (!x || !y) return SWIN_ERR_INVALID_ARG;
  const Range out[] = {{y, bytes, kActivation}}, in[] = {{x, bytes, kActivation}, state_of(d)};
  if (clash(out, in)) return SWIN_ERR_INVALID_ARG;
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
