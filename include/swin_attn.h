/*
 * swin_attn.h -- C ABI of a single-GPU (GB300, sm_103a) library for
 * shifted-window multi-head self-attention (SW-MSA) over a lat-lon(-depth)
 * token grid: cyclic shift, ragged edge windows, periodic longitude seam,
 * shift-boundary (region) mask, land mask, relative-position bias, softmax,
 * PV and the reverse routing back to the grid; forward and backward.
 *
 * Where the operation is defined (page title, section):
 *  - "TERRA: A Hierarchical Parallel Training and Memory Orchestration
 *    Framework for High-Resolution AI-based Earth Modeling", Sec. IV.D
 *    "Differentiable Token Routes": window coordinate and in-window offset of
 *    a token follow from its global grid coordinate; a window shift changes
 *    the coordinate; the backward applies the inverse route. Sec. V.A, Eq. (4):
 *    ragged contiguous window ranges (used here to split work over CTAs).
 *  - "4D Parallelism Unlocks Exascale Bayesian Neural Networks for
 *    High-Fidelity Atmospheric Modeling", Model Architecture: the domain is
 *    rolled by floor(window/2) between attention layers; Swin-style window
 *    attention with a relative-position bias.
 *
 * Definition computed (all dims outermost first; G grid, w window, s shift):
 *   rolled position p_d = (u_d - s_d) mod G_d of the token at coordinate u;
 *   window floor(p_d / w_d), slot p_d mod w_d (ceil(G_d / w_d) windows per dim,
 *   the last one may be short: its missing slots are pads);
 *   region bit d = [dim d not periodic and s_d > 0 and p_d >= G_d - s_d];
 *   key j is visible to query i iff same window, same region bits, j not land;
 *   s_ij = hd^-1/2 q_i.k_j + bias[row(i,j), h],
 *   row(i,j) = sum_d (sig_i,d - sig_j,d + w_d - 1) * prod_{e>d} (2 w_e - 1);
 *   O_i = softmax over visible j of s_ij, times V; land queries give O = 0.
 *
 * Conventions for every entry point:
 *  - Returns SWIN_OK (0) or a negative status; nothing is launched when an
 *    argument check fails.
 *  - Tensors are owned by the caller, device-resident, contiguous. Every
 *    q/k/v/o/dout/dq/dk/dv pointer and lse must be 16-byte aligned, land,
 *    bias and dbias 4-byte aligned: the tensor-core kernels read four
 *    consecutive LSE values, or land bytes, with one load. fwd and bwd
 *    return SWIN_ERR_ALIGNMENT (launching nothing) for any pointer that
 *    breaks this rule; buffer sizes are the caller's to keep.
 *  - q, k, v, o, dout, dq, dk, dv: [B, grid..., C] channel-last, C = heads *
 *    head_dim, head h in channels [h*hd, (h+1)*hd); element type = desc.dtype.
 *  - bias, dbias: float32 [rows][heads], rows = prod(2 w_d - 1).
 *  - lse: float32 [B][heads][grid...] natural-log log-sum-exp per query
 *    (-inf for land queries).
 *  - land: uint8 [B, grid...], nonzero = land.
 *  - fwd/bwd allocate nothing and are asynchronous on `stream`.
 */
#ifndef SWIN_ATTN_H
#define SWIN_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define SWIN_OK 0
#define SWIN_ERR_INVALID_ARG (-1) /* NULL/inconsistent argument or descriptor */
#define SWIN_ERR_UNSUPPORTED (-2) /* head_dim not 16/32/128, window too large for head_dim, ... */
#define SWIN_ERR_ALIGNMENT (-3)   /* a pointer breaks its alignment rule (see Conventions) */
#define SWIN_ERR_WORKSPACE (-4)   /* workspace NULL or smaller than required */
#define SWIN_ERR_CUDA (-5)        /* a CUDA runtime call or launch failed */
#define SWIN_ERR_TIMEOUT (-6)     /* a kernel gave up a bounded wait (device status word) */
#define SWIN_ERR_DEVICE (-7)      /* a kernel recorded another device-side error */

/* Element types of q, k, v, o, dout, dq, dk, dv. */
#define SWIN_F32 0
#define SWIN_BF16 1

/* Kernel family. AUTO picks the tensor-core path for bf16 with head_dim 32 or 128. */
#define SWIN_IMPL_AUTO 0
#define SWIN_IMPL_SIMT 1   /* fp32 FFMA kernels (head_dim 16/32, windows up to 128 slots) */
#define SWIN_IMPL_TC 2     /* tcgen05/TMEM kernels (bf16; head_dim 32 with windows up to 128
                              slots, or head_dim 128 with windows of any size) */

/* Same type as cudaStream_t; NULL is the legacy default stream. */
typedef struct CUstream_st *swin_stream_t;

/* Opaque plan. Owns its device-side tables and status word. */
typedef struct swin_attn_plan_s *swin_attn_plan_t;

typedef struct {
  int32_t ndim;        /* 2: (lat, lon); 3: (depth, lat, lon) */
  int32_t impl;        /* SWIN_IMPL_* */
  int64_t batch;       /* B >= 1 */
  int32_t grid[3];     /* G_d >= 1, outermost first; batch * prod(G) < 2^31 */
  int32_t window[3];   /* w_d >= 1; prod(w) <= 128, or <= 65536 with head_dim 128 */
  int32_t shift[3];    /* 0 <= s_d < w_d, s_d < G_d (or 0); all zero = W-MSA */
  int32_t periodic[3]; /* 1 = cyclic neighbour (no region bit), 0 = region-masked */
  int32_t heads;       /* >= 1 */
  int32_t head_dim;    /* 16 or 32; or 128 (bf16, tensor cores): windows of any size, split
                          into 128-slot query and key tiles with an online softmax */
  int32_t dtype;       /* SWIN_F32 or SWIN_BF16 */
  int32_t has_land;    /* 1 = a land mask is passed to fwd/bwd */
} swin_attn_desc;

/* Sizes and launch shapes of a plan (all counts, no pointers). */
typedef struct {
  int64_t windows_per_image;
  int64_t tokens_per_image;
  int32_t slots;       /* n = prod(w) */
  int32_t bias_rows;   /* prod(2 w_d - 1) */
  int32_t impl;        /* resolved SWIN_IMPL_SIMT or SWIN_IMPL_TC */
  int32_t fwd_ctas;    /* persistent CTAs of the forward kernel */
  int32_t bwd_ctas;    /* persistent CTAs of the backward kernel */
  int32_t num_sms;
  int64_t work_items;  /* heads * B * ceil(windows_per_image / k): one head and k windows each, k = 2 on
                          the tensor-core path when two windows fit one 128-slot tile, else 1 */
  int64_t dbias_slots; /* partial dBias tables in the workspace */
} swin_attn_plan_info;

/* Dropout decisions: Philox4x32-7 with key = seed and counter = (block low 32,
 * block high 32, site, step). Decision i is 16-bit number i % 8 of block
 * i / 8 (word (i % 8) / 2, low half first); it keeps iff that number is
 * >= T = rint(rate * 65536), and what is kept is multiplied by
 * 1 / (1 - T / 65536). What is dropped is 0 whatever it was (infinities and
 * NaN too). The backward passes recompute the decisions: give them the same
 * descriptor and an unchanged state. The state is read on the device when the
 * kernel runs, so a captured call replays with the state's current step. Sites
 * separate the dropouts of one step: two calls with one site, seed and step
 * drop the same positions. */
typedef struct {
  double rate;           /* 0 (none) <= rate, T <= 65535 */
  uint32_t site;
  const uint64_t *state; /* device, 8-byte aligned: {seed, step}; the step counts modulo 2^32.
                            May be NULL when the rate is 0 */
} swin_attn_drop;

/* Validate `desc` and build a plan on the current CUDA device: routing tables
 * (win_src, region, tok_dst, relidx) are computed on the device by the same
 * routing function the kernels use, and the work partition is fixed.
 * Synchronous; allocates device memory owned by the plan.
 * Errors: INVALID_ARG (NULL, bad sizes, shift >= window), UNSUPPORTED
 * (slots > 128 without head_dim 128, slots > 65536, head_dim, dtype, impl not
 * available for the dtype or head_dim), CUDA. */
int swin_attn_plan(const swin_attn_desc *desc, swin_attn_plan_t *out);

/* Copy `plan`'s sizes into *info (host). Errors: INVALID_ARG. */
int swin_attn_plan_get_info(swin_attn_plan_t plan, swin_attn_plan_info *info);

/* Copy the routing tables of one image to HOST buffers (any may be NULL):
 *   win_src [nwin][n] int32: grid token feeding slot s of window w, -1 = pad;
 *   region  [nwin][n] uint8: region bits of that token (bit d for dim d), 0 for pads;
 *   tok_dst [N] int32: w*n + s of every token (the inverse route);
 *   relidx  [n][n] int32: bias row of the slot pair (query i, key j); kept by
 *           the plan for windows of up to 2048 slots only (UNSUPPORTED above).
 * Synchronous. Errors: INVALID_ARG, UNSUPPORTED, CUDA. */
int swin_attn_plan_tables(swin_attn_plan_t plan, int32_t *win_src, uint8_t *region,
                          int32_t *tok_dst, int32_t *relidx);

/* Bytes of device workspace swin_attn_bwd needs: the partial dBias tables,
 * and for head_dim 128 also delta_i = sum_j P_ij dP_ij of every query. */
size_t swin_attn_workspace_bytes(swin_attn_plan_t plan);

/* Forward. q, k, v, o as above; bias may be NULL (zero bias); land required
 * iff desc.has_land; lse may be NULL (inference) else receives the float32
 * log-sum-exp. Pad slots write nothing; every grid token is written once.
 * head_dim 128: a non-NULL bias needs at most 4096 bias rows (UNSUPPORTED).
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, CUDA (launch). */
int swin_attn_fwd(swin_attn_plan_t plan, const void *q, const void *k, const void *v,
                  const float *bias, const uint8_t *land, void *o, float *lse,
                  swin_stream_t stream);

/* Backward of L = sum(O * dout): writes dq, dk, dv (every token) and
 * OVERWRITES dbias (may be NULL: not computed). lse is the forward's output
 * for the same inputs (required). delta_i = sum_j P_ij dP_ij is recomputed
 * in-kernel, so O is not an input. workspace: device, >=
 * swin_attn_workspace_bytes(plan) bytes, 256-byte aligned, contents ignored
 * (not needed when dbias is NULL, except with head_dim 128, whose backward
 * keeps delta there). head_dim 128: a non-NULL bias needs at most 4096 bias
 * rows and a non-NULL dbias at most 8192 (UNSUPPORTED); its dBias is summed
 * per CTA with shared-memory atomic adds, so it may differ between calls in
 * the last bits (the other outputs, and dBias of head_dim 16/32, do not).
 * When swin_attn_status then reports SWIN_ERR_TIMEOUT, every output of the
 * call is undefined.
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
int swin_attn_bwd(swin_attn_plan_t plan, const void *q, const void *k, const void *v,
                  const void *dout, const float *lse, const float *bias,
                  const uint8_t *land, void *dq, void *dk, void *dv, float *dbias,
                  void *workspace, size_t workspace_bytes, swin_stream_t stream);

/* Backward that also receives the forward's output o (same type, layout and
 * alignment as q; o of the same inputs). With head_dim 128, delta_i is then
 * sum over the head's channels of dout_ic * o_ic (FlashAttention's form of
 * the softmax derivative's row sum, which TERRA's FlashAttention backward
 * uses), computed by a small kernel before the query-tile kernel, which then
 * sweeps the key tiles once instead of twice. It differs from swin_attn_bwd's
 * delta by the rounding of o to the storage type. Other head dims ignore o
 * (their kernels recompute delta in the pass that needs it at no extra cost)
 * and give swin_attn_bwd's results. Other arguments, results and errors as
 * swin_attn_bwd; o NULL is INVALID_ARG, misaligned ALIGNMENT. */
int swin_attn_bwd_o(swin_attn_plan_t plan, const void *q, const void *k, const void *v, const void *o,
                    const void *dout, const float *lse, const float *bias, const uint8_t *land, void *dq,
                    void *dk, void *dv, float *dbias, void *workspace, size_t workspace_bytes,
                    swin_stream_t stream);

/* swin_attn_fwd with dropout of the probabilities (drop NULL or rate 0: none):
 *   O_i = sum over visible j of keep_ij / kept * softmax_ij * V_j;
 * the log-sum-exp is the softmax's, without dropout. Decision of query token
 * t (of image b, head h) and key slot j of its window of n slots:
 * 8 * (r * ceil(n / 8)) + j with r = (b * heads + h) * tokens + t.
 * Errors: those of swin_attn_fwd. */
int swin_attn_fwd_dropout(swin_attn_plan_t plan, const void *q, const void *k, const void *v, const float *bias,
                          const uint8_t *land, void *o, float *lse, const swin_attn_drop *drop,
                          swin_stream_t stream);

/* Its backward: with the same drop (and unchanged state) as the forward.
 *   dP_ij = keep_ij / kept * (dO_i . V_j), dS_ij = P_ij (dP_ij - sum_j P_ij dP_ij),
 *   dV_j = sum_i keep_ij / kept * P_ij dO_i.
 * o, the forward's output, may be NULL. Other arguments, results and errors as
 * swin_attn_bwd. */
int swin_attn_bwd_dropout(swin_attn_plan_t plan, const void *q, const void *k, const void *v, const void *o,
                          const void *dout, const float *lse, const float *bias, const uint8_t *land, void *dq,
                          void *dk, void *dv, float *dbias, void *workspace, size_t workspace_bytes,
                          const swin_attn_drop *drop, swin_stream_t stream);

/* Backward for callers that cannot allocate device memory. No counterpart on
 * the pages: it exists for callers whose host code has no device allocator
 * of its own (for example a C or Fortran model that only receives tensors),
 * or whose device memory all belongs to a pool they may not touch while
 * stepping, and who therefore cannot provide swin_attn_bwd's workspace.
 * Same arguments, results and errors as swin_attn_bwd without the
 * workspace: the partial dBias tables go to a fixed device array inside this
 * library (SWIN_NOALLOC_MAX_WORKSPACE_BYTES, held on every GPU that loads the
 * library until the process exits). Nothing is allocated by any call.
 *  - With dbias != NULL, plans whose swin_attn_workspace_bytes() exceeds
 *    the array are rejected with SWIN_ERR_WORKSPACE (nothing is launched).
 *    With dbias == NULL the array is not used and any plan is accepted.
 *  - The first call in a CUDA context (per device, and again after
 *    cudaDeviceReset or in another context on that device) looks up the
 *    array's device address in that context; make that first call before
 *    any stream capture.
 *  - All calls share the one array: calls that can overlap on the GPU (other
 *    streams, other threads) race on it; serialise them. Each call writes
 *    every partial table it reads; when swin_attn_status reports
 *    SWIN_ERR_TIMEOUT, that call's outputs (dbias included) are undefined.
 * Errors: those of swin_attn_bwd, WORKSPACE as above, CUDA. */
#define SWIN_NOALLOC_MAX_WORKSPACE_BYTES ((size_t)4 << 20)
int swin_attn_bwd_noalloc(swin_attn_plan_t plan, const void *q, const void *k, const void *v,
                          const void *dout, const float *lse, const float *bias,
                          const uint8_t *land, void *dq, void *dk, void *dv, float *dbias,
                          swin_stream_t stream);

/* The attention half of a Swin block in one kernel: LayerNorm and the QKV
 * projection as its prologue, SW-MSA as above, the out-projection and the
 * residual add as its epilogue, so that Q, K, V and O never go to device
 * memory (TERRA, Fig. 4 "Layernorm ... Window Attention ... MLP" and Sec. III;
 * BEAST page, "Model Architecture"). Per token t of image b:
 *   Xn = (x - mean) / sqrt(var + ln_eps) * ln_gamma + ln_beta
 *        (mean and biased variance over the C channels of x),
 *   [q | k | v] = bf16(Xn) W_qkv^T + b_qkv, each rounded to bf16,
 *   o = SW-MSA(q, k, v; bias, land) of the plan's geometry, rounded to bf16,
 *   y = x + o W_o^T + b_o, rounded to bf16.
 * x, y: bf16 [B, grid..., C], 16-byte aligned, y must not overlap x; every
 * grid token is written once. w_qkv: bf16 [3C][C] row-major (rows 0..C-1
 * give q, C..2C-1 k, 2C..3C-1 v; head h owns rows h*32..h*32+31 of each);
 * w_o: bf16 [C][C] row-major (row = output channel); both 16-byte aligned.
 * ln_gamma, ln_beta, b_o: float32 [C]; b_qkv: float32 [3C]; bias as above
 * (may be NULL); all 4-byte aligned. ln_eps > 0 and finite.
 * Supported plans: bf16, head_dim 32, at most 128 slots per window, C a
 * multiple of 64 up to 256, heads * bias rows <= 8192 (else UNSUPPORTED).
 * Forward only (no autograd through the projections here).
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, CUDA (launch). */
int swin_attn_block_fwd(swin_attn_plan_t plan, const void *x, const float *ln_gamma, const float *ln_beta,
                        float ln_eps, const void *w_qkv, const float *b_qkv, const void *w_o,
                        const float *b_o, const float *bias, const uint8_t *land, void *y,
                        swin_stream_t stream);

/* ---- Around the attention: norms, residual join, dropout -------------------
 * These work on rows of `channels` values, one row per token of
 * [images, tokens, channels] (the [B, grid..., C] tensors above with the grid
 * flattened); no plan is needed. They run on the current device, to which
 * every pointer must belong, allocate nothing and are asynchronous on
 * `stream`. Activations are 16-byte, float parameters 4-byte, workspaces
 * 256-byte aligned (ALIGNMENT). An activation may be written exactly over an
 * activation of the call, a parameter's gradient exactly over that parameter;
 * any other overlap of an output or the workspace with another output or an
 * input (a dropout's state too) is INVALID_ARG. With no rows nothing is read or written
 * but the parameter gradients, which are zero. All sums are fp32 in a fixed
 * order: the same inputs give the same bits. */

#define SWIN_NORM_NONE 0
#define SWIN_NORM_LAYER 1 /* (x - mean) / sqrt(var + eps), biased variance */
#define SWIN_NORM_RMS 2   /* x / sqrt(mean of squares + eps) */
typedef struct {
  int32_t kind;       /* SWIN_NORM_* */
  float eps;          /* > 0, finite */
  const float *gamma; /* [C]; NULL: ones */
  const float *beta;  /* [C]; NULL: zeros */
} swin_attn_norm;

typedef struct {
  int64_t images, tokens; /* >= 0; images * tokens < 2^31 (else UNSUPPORTED) */
  int32_t channels;       /* a multiple of 8, up to 8192 (else UNSUPPORTED) */
  int32_t dtype;          /* SWIN_F32 or SWIN_BF16: the activations' type */
} swin_attn_rows;

/* Bytes of device workspace the backward calls on these rows need for any
 * parameter gradient (0 for a bad descriptor). They grow with the images for
 * a gate alone: the norm and a join without a gate take the workspace of the
 * same rows as one image ({1, images * tokens}). */
size_t swin_attn_rows_workspace_bytes(const swin_attn_rows *rows);

/* The norm before a block: h = N(x). norm->kind is not NONE.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, CUDA. */
int swin_attn_norm_fwd(const swin_attn_rows *rows, const void *x, const swin_attn_norm *norm, void *h,
                       swin_stream_t stream);

/* Its backward: dx = dres + N^T dh (dres, the residual path's gradient, may be
 * NULL), and, where not NULL, dgamma = sum dh xhat and dbeta = sum dh [C]
 * (overwritten). The statistics are recomputed from x. The workspace is
 * needed for dgamma or dbeta only (WORKSPACE).
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
int swin_attn_norm_bwd(const swin_attn_rows *rows, const void *x, const swin_attn_norm *norm, const void *dh,
                       const void *dres, void *dx, float *dgamma, float *dbeta, void *workspace,
                       size_t workspace_bytes, swin_stream_t stream);

/* The residual join after a block whose output is z, with the next block's
 * norm:
 *   y = x + scale * gate * path * D(N_post(z)),   h = N_pre(y),
 * y rounded to the activations' type and h the norm of that stored y.
 * N_post and N_pre may be NONE (pre NONE: h is NULL). D: dropout of the
 * elements, element e of [images, tokens, C] being decision e. path: dropout
 * of whole images (stochastic depth), image b being decision b. */
typedef struct {
  swin_attn_norm post, pre;
  const float *scale; /* [C] layer scale; NULL: ones */
  const float *gate;  /* [images][C]; NULL: ones. Post-side parameter gradients beside a gate: up to
                         16 776 960 images (else UNSUPPORTED) */
  swin_attn_drop drop, path;
} swin_attn_join;

/* Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, CUDA. */
int swin_attn_join_fwd(const swin_attn_rows *rows, const void *x, const void *z, const swin_attn_join *join,
                       void *y, void *h, swin_stream_t stream);

/* Gradients of the join's parameters, each NULL where not wanted; gate is
 * [images][C], the others [C]. All are overwritten. */
typedef struct {
  float *post_gamma, *post_beta, *scale, *gate, *pre_gamma, *pre_beta;
} swin_attn_join_grads;

/* Backward of the join from its stored y (not x) and z: dx and dz. dy or dh
 * may be NULL (zero gradient), not both; y may be NULL when dh is, z when
 * there is no post norm and neither scale's nor gate's gradient is wanted.
 * The workspace is needed for parameter gradients only.
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
int swin_attn_join_bwd(const swin_attn_rows *rows, const void *y, const void *z, const swin_attn_join *join,
                       const void *dy, const void *dh, void *dx, void *dz, const swin_attn_join_grads *grads,
                       void *workspace, size_t workspace_bytes, swin_stream_t stream);

/* Dropout of n elements of type dtype: y_i = keep(i / span) ? x_i / kept : 0,
 * `span` consecutive elements sharing one decision (1: dropout; tokens * C:
 * stochastic depth per image). Its backward is the same call on the gradient.
 * n < 0 or above 2^46, or span < 1, is INVALID_ARG.
 * Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, CUDA. */
int swin_attn_dropout(int32_t dtype, int64_t n, int64_t span, const void *x, const swin_attn_drop *drop, void *y,
                      swin_stream_t stream);

/* ---- Between the projection and the attention: heads and their positions ----
 * The QKV projection leaves rows [q | k | v]; the attention takes q, k and v as
 * tensors of their own. These calls read up to four parts (of one packed tensor
 * or of several), norm every head, turn its values by the token's position, and
 * write each part where it is wanted, in one pass; and back. Per part, token and
 * head, with u = N(x) (gamma and beta [head_dim], shared by the part's heads):
 *   pair i of the first rotary.dim values of u, (a, b) = (u_i, u_{i + dim/2}) in the
 *   half layout, (u_2i, u_{2i+1}) in the interleaved one, becomes
 *   A (a cos t - b sin t), A (a sin t + b cos t) with t = position[axis_i] * f_i;
 *   the other values are u's.
 * Angles are kept in turns as 64-bit fixed point, freq_i = round(2^64 f_i / (2 pi))
 * modulo 2^64: a position times it wraps by itself, so the error of an angle is
 * |position| 2^-65 turns and no position is too far. Sums are fp32 in a fixed
 * order; each value is rounded once, when it is stored.
 * The rules of the rows' calls (above) hold: current device, nothing allocated,
 * asynchronous, alignments (rows' strides too: multiples of 16 bytes). A part's
 * output may lie exactly on its own x (forward), x or dy (backward), with the
 * same stride; any other overlap of an output with another output, an input or
 * the workspace is INVALID_ARG. Rows of one stride that lie side by side, as the
 * parts of a packed tensor do, do not overlap. */
#define SWIN_ROTARY_HALF 0
#define SWIN_ROTARY_INTERLEAVED 1
typedef struct {
  int32_t dim;           /* values of a head that turn: a multiple of 16 up to head_dim; 0: none */
  int32_t layout;        /* SWIN_ROTARY_* */
  float amplitude;       /* A, finite */
  const uint64_t *freq;  /* HOST [dim / 2], read by the call */
  const uint8_t *axis;   /* HOST [dim / 2], each below ndim */
  int32_t position_bits; /* 0: a token's grid coordinates are its positions; 32 or 64: they are given */
  int32_t shared;        /* given positions are 0: [images][tokens][ndim], 1: [tokens][ndim] of every image */
  const void *positions; /* device, int32 or int64 (aligned to them), any sign; NULL with grid coordinates */
} swin_attn_rotary;

typedef struct {
  int64_t images;   /* >= 0; images * tokens < 2^31 (else UNSUPPORTED) */
  int32_t ndim;     /* 1 to 3 */
  int32_t grid[3];  /* tokens of an image, outermost first, >= 0 */
  int32_t head_dim; /* a multiple of 16 up to 256 (else UNSUPPORTED) */
  int32_t dtype;    /* SWIN_F32 or SWIN_BF16 */
  swin_attn_rotary rotary;
} swin_attn_heads;

#define SWIN_HEAD_PARTS_MAX 4
typedef struct {
  int32_t heads;        /* 1 to 65535, heads * head_dim up to 16384 (else UNSUPPORTED) */
  int32_t rotate;       /* 0 or 1; neither this nor a norm: the part is copied */
  swin_attn_norm norm;  /* gamma, beta: [head_dim] */
  const void *x;        /* [images * tokens] rows of heads * head_dim values */
  int64_t x_stride;     /* elements from row to row, at least heads * head_dim */
  const void *dy;       /* backward: the gradient of the part's output (forward: ignored) */
  int64_t dy_stride;
  void *out;            /* forward: the part's output; backward: dx */
  int64_t out_stride;
  float *dgamma, *dbeta; /* backward: overwritten; NULL: not wanted. Not without a norm */
} swin_attn_head_part;

/* Forward of `count` parts. Errors: INVALID_ARG, ALIGNMENT, UNSUPPORTED, CUDA. */
int swin_attn_heads_fwd(const swin_attn_heads *heads, const swin_attn_head_part *parts, int32_t count,
                        swin_stream_t stream);

/* Bytes of device workspace that swin_attn_heads_bwd needs for dgamma and dbeta (0 for a bad descriptor). */
size_t swin_attn_heads_workspace_bytes(const swin_attn_heads *heads);

/* Backward: dx of every part, x being its forward's input (NULL for a part
 * without a norm: it is not read). The statistics are recomputed. The workspace
 * is needed for dgamma or dbeta only (WORKSPACE).
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
int swin_attn_heads_bwd(const swin_attn_heads *heads, const swin_attn_head_part *parts, int32_t count,
                        void *workspace, size_t workspace_bytes, swin_stream_t stream);

/* ---- After the backward: the parameters' step --------------------------------
 * One AdamW step over many tensors, and the global norm of their gradients. The
 * step count and the learning rate lie on the device and are read when the
 * kernels run, so a captured step replays with what it finds there.
 *   c = min(1, max_norm / |g|), |g| over all tensors of the call (c = 1 without max_norm),
 *   g' = c g, m = b1 m + (1 - b1) g', v = b2 v + (1 - b2) g'^2, t = steps so far + 1,
 *   w = w (1 - lr decay) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps).
 * A bf16 parameter is the rounded copy of an fp32 master weight. States are fp32,
 * or 8 bits: m and r = sqrt(v) in e4m3 times one fp32 scale of every 256
 * consecutive values of a tensor (the largest magnitude over 448), rounded to
 * nearest when stored (the step itself uses the unrounded ones); an r above 0 is
 * stored as 2^-9 of a scale at least, so that no denominator vanishes.
 * With max_norm, a gradient norm that is not finite (squares are fp32: magnitudes
 * above 1.8e19 count as infinite) leaves parameters, states and step count as
 * they are; without it, an element whose gradient is not finite becomes NaN, in 8
 * bits its 256 with it. Everything is fp32, sums in a fixed order: the same bits every run. */
typedef struct {
  int64_t n;         /* elements, >= 0 (0: skipped) */
  int32_t dtype;     /* of param: SWIN_F32 or SWIN_BF16 */
  int32_t grad_dtype;
  void *param;       /* updated */
  float *master;     /* SWIN_BF16: updated; NULL otherwise */
  const void *grad;  /* NULL: the tensor is skipped */
  void *m, *v;       /* [n] float, or bytes of e4m3 (v holds r) */
  float *m_scale, *v_scale; /* 8 bits: [ceil(n / 256)]; NULL otherwise */
  float decay;       /* weight decay, finite, >= 0 */
} swin_attn_param;

typedef struct {
  double beta1, beta2;  /* 0 <= beta < 1 */
  double eps;           /* > 0, finite */
  double max_norm;      /* > 0: clip; 0: do not */
  int32_t state_bits;   /* 32 or 8 */
  const float *lr;      /* device */
  int64_t *steps;       /* device: steps so far, counted up by the call */
  float *norm;          /* device, NULL: not wanted (with max_norm only): |g| before clipping */
} swin_attn_adamw;

/* Bytes of device workspace that the two calls below need. */
size_t swin_attn_adamw_workspace_bytes(void);

/* One step. Elements are aligned to their own size, the workspace to 256 bytes;
 * outputs (param, master, m, v, scales, steps, norm, workspace) overlap neither
 * one another nor any input (INVALID_ARG). All tensors' elements together, each
 * tensor's rounded up to 256: below 2^39 (else UNSUPPORTED).
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
int swin_attn_adamw_step(const swin_attn_adamw *adamw, const swin_attn_param *params, int64_t count,
                         void *workspace, size_t workspace_bytes, swin_stream_t stream);

/* norm = sqrt(sum of squares) of the gradients in params (n, grad, grad_dtype; the rest is ignored).
 * Errors: INVALID_ARG, ALIGNMENT, WORKSPACE, UNSUPPORTED, CUDA. */
int swin_attn_grad_norm(const swin_attn_param *params, int64_t count, float *norm, void *workspace,
                        size_t workspace_bytes, swin_stream_t stream);

/* Testing hook for the failure path of the tensor-core kernels (the fused
 * block's included). Every wait inside those kernels gives up after
 * `wait_limit_ns` (default 1 s) and then records SWIN_ERR_TIMEOUT in the
 * status word. force_timeout = 1 makes one role of the next launches wait on
 * a barrier that nothing arrives at, so the bounded wait runs out on purpose
 * (the kernel then drains and exits).
 * Errors: INVALID_ARG (NULL plan, zero limit, force_timeout not 0/1). */
int swin_attn_plan_set_debug(swin_attn_plan_t plan, uint64_t wait_limit_ns, int force_timeout);

/* Synchronise `stream`, read and clear the plan's device status word.
 * Returns SWIN_OK, SWIN_ERR_TIMEOUT, SWIN_ERR_DEVICE or SWIN_ERR_CUDA. */
int swin_attn_status(swin_attn_plan_t plan, swin_stream_t stream);

/* Free the plan's device memory (synchronises the device). NULL is a no-op. */
void swin_attn_plan_destroy(swin_attn_plan_t plan);

/* Static message for a status code. */
const char *swin_attn_strerror(int status);

/* TERRA Sec. V.A, Eq. (4): rank r of P ranks owns the contiguous window-index
 * range [floor(r*M/P), floor((r+1)*M/P)). Host-only, used for the CTA work
 * split. Errors: INVALID_ARG (M < 0, P < 1, r outside [0, P), NULL). */
int swin_attn_window_range(int64_t M, int64_t P, int64_t r, int64_t *L, int64_t *R);

/* TERRA Sec. V.A, Eq. (3): the fixed (two-dimensional round-robin) window
 * assignment over an m x n mesh pads each input dimension until every rank
 * owns the same number of whole windows. For one dimension of `extent` input
 * points, `stride` input points per token (patch size times sampling factor,
 * p*alpha), `window` tokens per window and `ranks` mesh ranks along that
 * dimension (m or n): *padded = ceil(extent / q) * q, q = stride*window*ranks.
 * ranks = 1 gives the least padding to whole windows, the padding that the
 * ragged assignment of Eq. (4) keeps. Host-only arithmetic; the attention
 * kernels never pad (pad slots of ragged windows are masked instead).
 * Errors: INVALID_ARG (extent, stride, window or ranks below 1, NULL, or a
 * result above INT64_MAX). */
int swin_attn_fixed_padded_extent(int64_t extent, int64_t stride, int64_t window, int64_t ranks,
                                  int64_t *padded);

#ifdef __cplusplus
}
#endif

#endif /* SWIN_ATTN_H */
