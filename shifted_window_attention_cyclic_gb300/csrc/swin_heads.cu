// swin_heads.cu -- between the QKV projection and the attention: the norm of every
// head and rotary positions, read from the projection's packed rows and written
// where the attention takes them; forward and backward (sm_103a).
//
//   u = N(x) gamma + beta over the head_dim values of a head,
//   (a, b) -> A (a cos t - b sin t, a sin t + b cos t), t = position[axis] f.
// Backward: du = A R(-t) dy, dgamma = sum du xhat, dbeta = sum du, g = du gamma,
//   dx = rstd (g - m(g) - xhat m(g xhat)), m the mean over the head (no m(g) for RMS).
// A part without a norm has no statistics: its backward is its forward at -t.
//
// Angles: a position times a frequency in turns, as 64-bit fixed point modulo one
// turn; the product wraps exactly, so there is no large argument to reduce, and a
// float takes the remaining fraction (2^-25 of a half turn off at most).
//
// What bounds them: HBM. Each value is read and written once (forward 1 179 648 x 24
// heads of 32, bf16, normed: 607 us, 6.0 TB/s, 89 % of the measured copy rate;
// 138 240 x 16 heads of 128 turned alone: 176 us, 96 %; their first form, with a vector
// a lane, shuffles and no loads ahead: 918 and 413 us).
#include <cmath>

#include "swin_heads.cuh"

namespace swin {
namespace {

using namespace heads;

// ---- parameter gradients from the CTAs' sums -----------------------------------
struct FoldArgs {
  int hd, count;
  Part parts[SWIN_HEAD_PARTS_MAX];
};

constexpr int kFoldLanes = 32;

// Block (tile, part): 32 channels, whose CTA sums 32 lanes add up in a fixed order.
__global__ void __launch_bounds__(32 * kFoldLanes) fold_kernel(const __grid_constant__ FoldArgs a) {
  // launched while the head kernel's last CTAs still run: their sums are there after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Part &p = a.parts[blockIdx.y];
  if (!p.dgamma && !p.dbeta) return;
  __shared__ float2 buf[kFoldLanes][33];
  const int tile = blockIdx.x * 32, c = min(tile + (int)threadIdx.x, a.hd - 1);
  float2 s = make_float2(0.f, 0.f);
  for (int i = threadIdx.y; i < p.ctas; i += kFoldLanes)
    s = add(s, make_float2(p.sums[(int64_t)i * 2 * a.hd + c], p.sums[((int64_t)i * 2 + 1) * a.hd + c]));
  buf[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = buf[threadIdx.x][threadIdx.y];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    s = add(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, o), __shfl_xor_sync(0xffffffffu, s.y, o)));
  const int mine = tile + (int)threadIdx.y;
  if (threadIdx.x == 0 && mine < a.hd) {
    if (p.dgamma) p.dgamma[mine] = s.x;
    if (p.dbeta) p.dbeta[mine] = s.y;
  }
}

// ---- argument checks -------------------------------------------------------------
// Rows of a tensor: `width` bytes every `stride`, or one stretch (rows = 1).
struct Span {
  const void *at;
  int64_t stride, width, rows;
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(at); }
  uintptr_t end() const { return begin() + (uintptr_t)((rows - 1) * stride + width); }
};
Span stretch(const void *at, int64_t bytes) { return {at, bytes, bytes, 1}; }

bool meet(const Span &a, const Span &b) {
  if (!a.at || !b.at || a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1) return false;
  if (a.begin() >= b.end() || b.begin() >= a.end()) return false;
  if (a.rows == 1 && b.rows == 1) return true;
  const int64_t stride = a.rows > 1 ? a.stride : b.stride;
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;  // (not told apart)
  // side by side within the stride?
  const uintptr_t gap = b.begin() >= a.begin() ? (b.begin() - a.begin()) % stride
                                               : (stride - (a.begin() - b.begin()) % stride) % stride;
  return !((int64_t)gap >= a.width && (int64_t)gap + b.width <= stride);
}
bool same(const Span &a, const Span &b) {
  return a.at == b.at && a.rows == b.rows && a.width == b.width && (a.stride == b.stride || a.rows == 1);
}

int check_heads(const swin_attn_heads *h, int64_t *rows, int64_t *tokens) {
  if (!h || h->images < 0 || h->ndim < 1 || h->ndim > 3) return SWIN_ERR_INVALID_ARG;
  if (h->dtype != SWIN_F32 && h->dtype != SWIN_BF16) return SWIN_ERR_UNSUPPORTED;
  if (h->head_dim < 16 || h->head_dim % 16 || h->head_dim > 256) return SWIN_ERR_UNSUPPORTED;
  if (h->images > INT32_MAX) return SWIN_ERR_UNSUPPORTED;
  bool none = h->images == 0;
  for (int a = 0; a < h->ndim; ++a) {
    if (h->grid[a] < 0) return SWIN_ERR_INVALID_ARG;
    none = none || h->grid[a] == 0;
  }
  *rows = *tokens = 0;
  if (!none) {
    int64_t n = 1;
    for (int a = 0; a < h->ndim; ++a)
      if ((n *= h->grid[a]) > INT32_MAX) return SWIN_ERR_UNSUPPORTED;
    *tokens = n;
    if ((*rows = n * h->images) > INT32_MAX) return SWIN_ERR_UNSUPPORTED;
  }
  const swin_attn_rotary &r = h->rotary;
  if (r.dim < 0 || r.dim % 16 || r.dim > h->head_dim) return SWIN_ERR_INVALID_ARG;
  if (r.dim == 0) return SWIN_OK;
  if (r.layout != SWIN_ROTARY_HALF && r.layout != SWIN_ROTARY_INTERLEAVED) return SWIN_ERR_INVALID_ARG;
  if (!std::isfinite(r.amplitude) || !r.freq || !r.axis) return SWIN_ERR_INVALID_ARG;
  for (int i = 0; i < r.dim / 2; ++i)
    if (r.axis[i] >= h->ndim) return SWIN_ERR_INVALID_ARG;
  if (r.position_bits != 0 && r.position_bits != 32 && r.position_bits != 64) return SWIN_ERR_INVALID_ARG;
  if (r.shared != 0 && r.shared != 1) return SWIN_ERR_INVALID_ARG;
  if (r.position_bits == 0 && r.positions) return SWIN_ERR_INVALID_ARG;
  return SWIN_OK;
}

// Values of a part's row: at most 10 chunks of a CTA's items (113 heads of 144, 12 at a time), which
// the workspace counts on.
constexpr int64_t kMostWidth = 16384;
constexpr int kMostChunks = 10;

int run(const swin_attn_heads *h, const swin_attn_head_part *parts, int count, bool bwd, void *workspace,
        size_t workspace_bytes, cudaStream_t st) {
  Args a = {};
  int64_t rows = 0, tokens = 0;
  int rc = check_heads(h, &rows, &tokens);
  if (rc) return rc;
  if (!parts || count < 1 || count > SWIN_HEAD_PARTS_MAX) return SWIN_ERR_INVALID_ARG;
  const int64_t e = h->dtype == SWIN_BF16 ? 2 : 4, cb = sizeof(float) * h->head_dim;
  const swin_attn_rotary &r = h->rotary;
  bool turns = false, norms = false, want = false;
  for (int i = 0; i < count; ++i) {
    const swin_attn_head_part &q = parts[i];
    if (q.heads < 1 || q.heads > 65535 || (q.rotate != 0 && q.rotate != 1)) return SWIN_ERR_INVALID_ARG;
    if ((int64_t)q.heads * h->head_dim > kMostWidth) return SWIN_ERR_UNSUPPORTED;
    if (q.norm.kind < SWIN_NORM_NONE || q.norm.kind > SWIN_NORM_RMS) return SWIN_ERR_INVALID_ARG;
    const bool norm = q.norm.kind != SWIN_NORM_NONE;
    if (norm && (!(q.norm.eps > 0.f) || !std::isfinite(q.norm.eps))) return SWIN_ERR_INVALID_ARG;
    if (!norm && (q.norm.gamma || q.norm.beta || (bwd && (q.dgamma || q.dbeta)))) return SWIN_ERR_INVALID_ARG;
    if (mis(q.norm.gamma, 4) || mis(q.norm.beta, 4) || (bwd && (mis(q.dgamma, 4) || mis(q.dbeta, 4))))
      return SWIN_ERR_ALIGNMENT;
    const int64_t width = (int64_t)q.heads * h->head_dim;
    const bool reads_x = !bwd || norm;
    const int64_t most = INT64_MAX / 4 / (rows + 1);  // bytes of a tensor stay below 2^63
    for (int k = 0; k < 3; ++k) {
      const int64_t stride = k == 0 ? q.x_stride : k == 1 ? q.dy_stride : q.out_stride;
      if ((k == 0 && !reads_x) || (k == 1 && !bwd) || rows < 2) continue;
      if (stride < width || stride > most) return SWIN_ERR_INVALID_ARG;
      if (stride * e % 16) return SWIN_ERR_ALIGNMENT;
    }
    if (rows) {
      if ((reads_x && !q.x) || (bwd && !q.dy) || !q.out) return SWIN_ERR_INVALID_ARG;
      if ((reads_x && mis(q.x, 16)) || (bwd && mis(q.dy, 16)) || mis(q.out, 16)) return SWIN_ERR_ALIGNMENT;
    }
    turns = turns || (q.rotate && r.dim);
    norms = norms || norm;
    want = want || (bwd && (q.dgamma || q.dbeta));
  }
  if (turns && r.position_bits && rows) {
    if (!r.positions) return SWIN_ERR_INVALID_ARG;
    if (mis(r.positions, r.position_bits / 8)) return SWIN_ERR_ALIGNMENT;
  }
  // overlaps: an output may lie on its own part's input, a gradient on its own parameter
  const Span ws = stretch(want ? workspace : nullptr, (int64_t)std::min<size_t>(workspace_bytes, INT64_MAX / 4));
  const Span at = stretch(turns && r.position_bits ? r.positions : nullptr,
                          (r.shared ? tokens : rows) * h->ndim * (r.position_bits / 8));
  struct Spans {
    Span x, dy, out, gamma, beta, dgamma, dbeta;
  } sp[SWIN_HEAD_PARTS_MAX];
  for (int i = 0; i < count; ++i) {
    const swin_attn_head_part &q = parts[i];
    const int64_t width = (int64_t)q.heads * h->head_dim * e;
    const bool reads_x = !bwd || q.norm.kind != SWIN_NORM_NONE;
    // (one row's stride is not looked at)
    auto rows_of = [&](const void *p, int64_t stride) { return Span{p, rows > 1 ? stride * e : width, width, rows}; };
    sp[i] = {rows_of(reads_x ? q.x : nullptr, q.x_stride),
             rows_of(bwd ? q.dy : nullptr, q.dy_stride),
             rows_of(q.out, q.out_stride),
             stretch(q.norm.gamma, cb),
             stretch(q.norm.beta, cb),
             stretch(bwd ? q.dgamma : nullptr, cb),
             stretch(bwd ? q.dbeta : nullptr, cb)};
  }
  for (int i = 0; i < count; ++i) {
    const Span outs[4] = {sp[i].out, sp[i].dgamma, sp[i].dbeta, i ? Span{} : ws};
    for (int o = 0; o < 4; ++o) {
      if (meet(outs[o], at)) return SWIN_ERR_INVALID_ARG;
      for (int p = o + 1; p < 4; ++p)
        if (meet(outs[o], outs[p])) return SWIN_ERR_INVALID_ARG;
      for (int j = 0; j < count; ++j) {
        const Spans &t = sp[j];
        if (j != i && (meet(outs[o], t.out) || meet(outs[o], t.dgamma) || meet(outs[o], t.dbeta)))
          return SWIN_ERR_INVALID_ARG;
        const Span *ins[4] = {&t.x, &t.dy, &t.gamma, &t.beta};
        for (int k = 0; k < 4; ++k) {
          const bool own = j == i && ((o == 0 && k < 2) || (o == 1 && k == 2) || (o == 2 && k == 3));
          if (meet(outs[o], *ins[k]) && !(own && same(outs[o], *ins[k]))) return SWIN_ERR_INVALID_ARG;
        }
      }
    }
  }
  if (want) {
    if (!workspace || workspace_bytes < swin_attn_heads_workspace_bytes(h)) return SWIN_ERR_WORKSPACE;
    if (mis(workspace, 256)) return SWIN_ERR_ALIGNMENT;
  }
  if (!rows) {
    for (int i = 0; i < count && bwd; ++i)
      for (float *d : {parts[i].dgamma, parts[i].dbeta})
        if (d && cudaMemsetAsync(d, 0, cb, st) != cudaSuccess) return SWIN_ERR_CUDA;
    return SWIN_OK;
  }

  int sms = 0;
  if ((rc = sm_count(&sms))) return rc;
  const bool stats = bwd && norms;  // else the backward is the forward at -t
  a.rows = (int)rows;
  a.hd = h->head_dim;
  a.ndim = h->ndim;
  a.count = count;
  a.layout = r.layout;
  a.amplitude = r.amplitude;
  a.positions = r.positions;
  a.position_bits = r.position_bits;
  a.shared = r.shared;
  a.by_tokens = FastDiv::by((uint32_t)tokens);
  if (turns) {
    a.pair_lanes = 8;
    while (a.pair_lanes < r.dim / 2) a.pair_lanes *= 2;
    uint32_t stride = 1;
    for (int d = h->ndim - 1; d >= 0; --d) {
      a.stride[d] = FastDiv::by(stride);
      a.extent[d] = FastDiv::by((uint32_t)h->grid[d]);
      stride *= (uint32_t)h->grid[d];
    }
    for (int i = 0; i < r.dim / 2; ++i) {
      a.freq[i] = bwd ? 0 - r.freq[i] : r.freq[i];
      a.axis[i] = r.axis[i];
    }
  }
  const int lanes = lanes_of(a.hd);
  const int threads = threads_of(stats), items = threads / lanes * items_of((int)e);
  const int64_t most = (int64_t)sms * kBlocks;
  int64_t bytes[SWIN_HEAD_PARTS_MAX], tiles[SWIN_HEAD_PARTS_MAX], all = 0, tiles_all = 0;
  bool beta = false;
  for (int i = 0; i < count; ++i) {
    const swin_attn_head_part &q = parts[i];
    Part &p = a.parts[i];
    p.chunks = (q.heads + items - 1) / items;
    p.by_heads = FastDiv::by((uint32_t)(p.chunks > 1 ? items : q.heads));
    p.tile_rows = std::max(1, items / q.heads);
    bytes[i] = q.heads * (int64_t)(stats && q.norm.kind != SWIN_NORM_NONE ? 3 : 2);
    tiles[i] = (rows + p.tile_rows - 1) / p.tile_rows * p.chunks;
    all += bytes[i];
    tiles_all += tiles[i];
    beta = beta || (bwd ? q.dbeta != nullptr : q.norm.beta != nullptr);
  }
  int ctas = 0;
  float *sums = static_cast<float *>(workspace);
  FoldArgs fold = {};
  for (int i = 0; i < count; ++i) {
    const swin_attn_head_part &q = parts[i];
    Part &p = a.parts[i];
    const bool norm = q.norm.kind != SWIN_NORM_NONE, as_x = bwd && !stats;
    p.x = static_cast<const uint8_t *>(as_x ? q.dy : q.x);
    p.x_stride = (as_x ? q.dy_stride : q.x_stride) * e;
    p.dy = static_cast<const uint8_t *>(q.dy);
    p.dy_stride = q.dy_stride * e;
    p.out = static_cast<uint8_t *>(q.out);
    p.out_stride = q.out_stride * e;
    p.heads = q.heads;
    p.kind = q.norm.kind;
    p.rot = q.rotate ? r.dim : 0;
    p.eps = q.norm.eps;
    p.gamma = q.norm.gamma;
    p.beta = q.norm.beta;
    p.wide_x = !mis(p.x, 32) && (rows < 2 || p.x_stride % 32 == 0);
    p.wide_dy = !mis(p.dy, 32) && (rows < 2 || p.dy_stride % 32 == 0);
    p.wide_out = !mis(p.out, 32) && (rows < 2 || p.out_stride % 32 == 0);
    // CTAs by the bytes a part moves, all resident at once; whole sets of a row's chunks
    p.cta0 = ctas;
    const int64_t share = tiles_all <= most ? tiles[i] : std::min(tiles[i], most * bytes[i] / all);
    p.ctas = (int)std::max<int64_t>(1, share / p.chunks) * p.chunks;
    ctas += p.ctas;
    if (bwd && norm && (q.dgamma || q.dbeta)) {
      p.sums = sums;
      p.dgamma = q.dgamma;
      p.dbeta = q.dbeta;
      sums += (int64_t)p.ctas * 2 * a.hd;
    }
    if (p.rot) a.table = std::max(a.table, p.tile_rows * table_row(p.rot >> 4));
    fold.parts[i] = p;
  }
  size_t smem = (size_t)a.table * 2 * sizeof(float);
  if (stats) smem = std::max(smem + kParamFloats * sizeof(float), (size_t)(threads / 32) * 2 * lanes * 16 * sizeof(float));
  rc = h->dtype == SWIN_BF16 ? launch_bf16(a, stats, norms, beta, ctas, smem, st)
                             : launch_f32(a, stats, norms, beta, ctas, smem, st);
  if (rc || !want) return rc;
  fold.hd = a.hd;
  fold.count = count;
  return launch_dependent(fold_kernel, dim3((a.hd + 31) / 32, count), dim3(32, kFoldLanes), 0, st, fold);
}

}  // namespace
}  // namespace swin

using namespace swin;

extern "C" {

size_t swin_attn_heads_workspace_bytes(const swin_attn_heads *h) {
  int64_t rows = 0, tokens = 0;
  int sms = 0;
  if (check_heads(h, &rows, &tokens) || sm_count(&sms)) return 0;
  const size_t need = ((size_t)sms * kBlocks + SWIN_HEAD_PARTS_MAX * kMostChunks) * 2 * h->head_dim * sizeof(float);
  return (need + 255) & ~size_t(255);
}

int swin_attn_heads_fwd(const swin_attn_heads *heads, const swin_attn_head_part *parts, int32_t count,
                        swin_stream_t stream) {
  return run(heads, parts, count, false, nullptr, 0, static_cast<cudaStream_t>(stream));
}

int swin_attn_heads_bwd(const swin_attn_heads *heads, const swin_attn_head_part *parts, int32_t count,
                        void *workspace, size_t workspace_bytes, swin_stream_t stream) {
  return run(heads, parts, count, true, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
