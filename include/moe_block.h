/*
 * moe_block.h -- C ABI of the operators around and beside the MI355X (gfx950)
 * sparse MoE layer: other selection rules for its router with their gradient,
 * its experts in 8-bit integers, and the norms before and after a block with
 * the block's gate and the residual's scale.  Same library, status codes,
 * types and layer shape as moe.h.
 *
 * Conventions (as in moe.h, with what differs stated at each call)
 *   - Pointers to arrays are DEVICE pointers owned by the caller; scratch
 *     comes from `ws`.  The library allocates, frees and keeps nothing after
 *     the call returns.  `stream` is a hipStream_t of the current device
 *     (NULL = the default stream); calls only enqueue work and can be
 *     captured into a HIP graph.  A workspace serves one call at a time: two
 *     calls, or two graphs, that may overlap need one each.
 *   - Return value: MOE_OK (0) or a negative moe_status.  Arguments are
 *     checked on the host before anything is enqueued.  Offsets, expert ids
 *     and permutations in device memory cannot be: the kernels keep every row
 *     that they name inside the arrays, so wrong ones give wrong values and
 *     never an access out of range (the debug build reports them,
 *     moe_debug_checks).  An array that is written must not overlap any other
 *     of the call (MOE_EINVAL) but where the call says that it may be another's
 *     memory.
 *   - Sums are formed in a fixed order, without atomics: the same call gives
 *     the same bits.
 */
#ifndef MOE_MI355X_BLOCK_H
#define MOE_MI355X_BLOCK_H

#include "moe.h"
#include "moe_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- selection of experts ------------------------------------------------ */

typedef enum {
  MOE_SCORE_SOFTMAX = 0, /* p = softmax(logits) over all experts */
  MOE_SCORE_SIGMOID = 1  /* p = 1 / (1 + exp(-logits))           */
} moe_score;

/* How experts are selected (host struct, copied into the launch).
 * Limits: n_groups >= 1 divides E; 1 <= top_groups <= n_groups <= 64;
 * group_best 1 or 2, at most E / n_groups; top_k <= top_groups * E / n_groups;
 * renorm_eps >= 0 and finite. */
typedef struct {
  int32_t score;      /* moe_score                                           */
  int32_t n_groups;   /* groups of E / n_groups neighbouring experts         */
  int32_t top_groups; /* groups that a token may select from                 */
  int32_t group_best; /* a group's score is the sum of its 1 or 2 best keys  */
  int32_t renorm;     /* nonzero: gates are divided by their sum             */
  float renorm_eps;   /* added to that sum                                   */
} moe_select_params;

/* moe_select -- scores, group-limited top-k by biased key, and gates, from
 * the router's logits (moe_route's selection is the case softmax, one group,
 * no renormalisation).  E = n_ffn + n_zero; of `shape`, T, n_ffn, n_zero,
 * top_k and routed_scaling matter.
 *   p[t, :]   = score(logits[t, :])
 *   key[t, e] = p[t, e] + bias[e]            (bias NULL: 0)
 *   the top_groups groups with the largest sums of their group_best largest
 *   keys stay (ties -> lower group), of their experts the top_k largest keys
 *   are taken (ties -> lower id) and written in ascending id:
 *   topk_idx[t, :]  [T, top_k] int32
 *   topk_gate[t, j] = routed_scaling f_j      [T, top_k] fp32
 *   f_j = p[t, idx_j], or with renorm p[t, idx_j] / (sum_i p[t, idx_i] +
 *         renorm_eps) (0 where that divisor is 0)
 * The selection is that of keys computed in 64 bits: keys too close for fp32
 * to tell apart are computed again.  Scores and gates are fp32, scores below its
 * normal numbers 0, but where a renormalised gate's divisor is below 2^-64: there
 * they count as 64 bits hold them.
 *   logits [T, E] fp32, E <= ld_logits < 2^24 elements from row to row; bias
 *   [E] fp32.  Shape limits as in moe.h, and T * top_k < 2^27 (here and in the
 *   calls below that take moe_select_params).
 * An expert with bias -inf is taken only where the kept groups have fewer than
 * top_k others, and does not count in its group's sum; one with +inf comes
 * before all others, its group before other groups.  A NaN key ranks as -inf.  A
 * logit of -inf has p = 0, also in a row that holds nothing else; a softmax over a
 * row with a NaN or +inf is NaN throughout.  Experts are switched off with -inf: a
 * finite bias far beyond all scores costs every token the 64-bit keys (fp32 cannot
 * tell what it is added to).  Any alignment of 4 bytes. */
int moe_select(const moe_shape* shape, const moe_select_params* params, const float* logits,
               int64_t ld_logits, const float* bias, int32_t* topk_idx, float* topk_gate,
               void* stream);

/* moe_route_select -- moe_route with another selection rule: the router's
 * product, then moe_select on its logits.
 *   logits_out [T, E] fp32: written, needed; ws: moe_workspace_bytes(shape);
 *   otherwise as moe_route (bias may be NULL). */
int moe_route_select(const moe_shape* shape, const moe_select_params* params, const void* x,
                     const void* w_router, const float* logit_bias, const float* bias,
                     int32_t* topk_idx, float* topk_gate, float* logits_out, void* ws,
                     void* stream);

/* moe_select_backward -- gradient at the logits from the gradient at the
 * gates.  With D = sum_i p_i + renorm_eps over the slots' experts:
 *   dp_j = routed_scaling dgate_j, or with renorm
 *          routed_scaling (dgate_j - sum_i dgate_i f_i) / D
 *   dlogits[t, e] = p_e (dp_e - sum_j p_j dp_j)   softmax
 *                 = p_e (1 - p_e) dp_e            sigmoid
 * dp_e being the sum over the slots that name e (more than one only in a
 * selection that moe_select did not make), 0 for other experts.  Selection
 * and bias have no gradient.  A slot whose id is outside [0, E) counts as an
 * expert of score 0.
 *   logits [T, E] fp32, ld_logits as there; topk_idx, dgate [T, top_k];
 *   dlogits [T, E] fp32, contiguous. */
int moe_select_backward(const moe_shape* shape, const moe_select_params* params,
                        const float* logits, int64_t ld_logits, const int32_t* topk_idx,
                        const float* dgate, float* dlogits, void* stream);

/* moe_layer_backward_select -- moe_layer_backward of a layer whose experts
 * moe_select chose: the same, with dlogits as moe_select_backward gives it.
 * io->logits is needed; ws: moe_layer_backward_workspace_bytes(shape).  Overlaps
 * are refused here, which moe_layer_backward leaves to its caller. */
int moe_layer_backward_select(const moe_shape* shape, const moe_select_params* params,
                              const moe_backward_io* io, void* ws, void* stream);

/* ---- products in 8-bit integers ------------------------------------------ */

/* Rows to quantise: x [M, K], ldx elements from row to row, q [M, K] with
 * ldq.  Limits: 0 <= M < 2^27; 1 <= K < 2^17; K <= ldx, ldq < 2^24. */
typedef struct {
  int32_t dtype; /* moe_dtype of x */
  int32_t M, K;
  int32_t reserved; /* 0 */
  int64_t ldx, ldq;
} moe_quant_shape;

/* moe_quantize_rows -- 8-bit codes with a scale for each row (weights: one
 * row is one output channel):
 *   scale[m] = max(max_k |x[m, k]| / 127, 2^-126)     fp32, rounded once
 *   q[m, k]  = the whole number nearest to x[m, k] / scale[m] (the exact
 *              quotient, ties to even), within [-127, 127]
 * A row that holds an infinity or a NaN has scale NaN and codes 0.  16-byte
 * aligned x and q, scale 4; any strides. */
int moe_quantize_rows(const moe_quant_shape* shape, const void* x, int8_t* q, float* scale,
                      void* stream);

/* Sizes of a product of 8-bit rows and weights, grouped by expert.
 *   a [M, K] int8 with lda elements from row to row, W [n_groups, N, K] int8
 *   and its scales [n_groups, N] contiguous, c [M, N] with ldc.
 * Limits: 1 <= n_groups <= 1024; 0 <= M < 2^27; 1 <= N <= 2^20; 1 <= K < 2^17
 * (a sum of K products of codes stays inside 32 bits); K <= lda < 2^24;
 * N <= ldc < 2^24.  Any sizes and strides within them; the fast kernels take K
 * and lda that are multiples of 16 with N and ldc that are multiples of 4, and
 * lda and ldc up to 2^20. */
typedef struct {
  int32_t out_dtype; /* moe_dtype of c                                       */
  int32_t n_groups;
  int32_t M;         /* rows that a and c have room for; the tiles go by it  */
  int32_t N, K;
  int32_t reserved;  /* 0                                                    */
  int64_t lda, ldc;
} moe_i8_shape;

/* Bytes of `ws` that moe_matmul_i8 needs for `shape` on the current device
 * (partial sums of products whose reduction is split to fill the chip; 0 for
 * most shapes, then ws may be NULL).  0 too if the shape is invalid. */
size_t moe_matmul_i8_workspace_bytes(const moe_i8_shape* shape);

/* moe_matmul_i8 -- c[p, n] = (sum_k a[p, k] W_e[n, k]) a_scale[p] w_scale[e, n]
 * for the rows p of group e, offsets[e] <= p < offsets[e + 1].
 *   offsets [n_groups + 1] int32, ascending, or NULL with one group: all M
 *   rows.  Rows behind offsets[n_groups] are neither read nor written.
 * The sum is exact in 32 bits whatever the codes (-128 too); it is converted
 * to fp32 once, multiplied by a_scale, then by w_scale, and rounded to
 * out_dtype.  16-byte aligned a, W, c; offsets
 * and scales 4; a, a_scale and c may be NULL when M = 0. */
int moe_matmul_i8(const moe_i8_shape* shape, const int32_t* offsets, const int8_t* a,
                  const float* a_scale, const int8_t* w, const float* w_scale, void* c, void* ws,
                  void* stream);

/* Arrays of the experts' FFN in 8-bit integers (a host struct of device
 * pointers, read during the call). */
typedef struct {
  const void* x;          /* [T, d_model] dtype; NULL where xq is given        */
  const int8_t* xq;       /* [T, d_model] codes of x (moe_quantize_rows,       */
  const float* x_scale;   /* [T]           moe_norm_residual), or both NULL    */
  const int32_t* perm;    /* [T * top_k]                                       */
  const int32_t* offsets; /* [E + 1]                                           */
  const int8_t* w_gate;   /* [n_ffn, d_ff, d_model]                            */
  const int8_t* w_up;     /* [n_ffn, d_ff, d_model]                            */
  const int8_t* w_down;   /* [n_ffn, d_model, d_ff]                            */
  const float* s_gate;    /* [n_ffn, d_ff]     scale of each output channel    */
  const float* s_up;      /* [n_ffn, d_ff]                                     */
  const float* s_down;    /* [n_ffn, d_model]                                  */
  void* y_perm;           /* [T * top_k, d_model] dtype: rows < offsets[n_ffn] */
} moe_ffn_i8_io;

/* Bytes of `ws` that moe_expert_ffn_i8 needs for `shape` on the current
 * device; 0 if the shape is invalid. */
size_t moe_expert_ffn_i8_workspace_bytes(const moe_shape* shape);

/* moe_expert_ffn_i8 -- moe_expert_ffn with 8-bit weights and rows: for the
 * sorted assignment p of expert e, x's row perm[p] / top_k
 *   xq, sx = moe_quantize_rows(x)   (once per token)
 *   z = (xq Wg^T) sx sg,  u = (xq Wu^T) sx su,  H = silu(z) u rounded to dtype
 *   hq, sh = moe_quantize_rows(H)
 *   y_perm[p] = (hq Wd^T) sh sd     rounded to dtype
 * sums exact; z, u and silu in fp32 where dtype is bf16, in 64 bits where it
 * is fp32 (an fp32 H decides the next code).  Shape limits as in moe.h, and
 * T * top_k < 2^27, d_model and d_ff < 2^17, T * d_model < 2^31 - 2^16. */
int moe_expert_ffn_i8(const moe_shape* shape, const moe_ffn_i8_io* io, void* ws, void* stream);

/* ---- norms around a block ------------------------------------------------ */

/* One residual step.  Limits: 0 <= T < 2^27; 1 <= d_model <= 32768;
 * rows_per_gate >= 1; eps >= 0 and finite, res_scale finite. */
typedef struct {
  int32_t T, d_model;
  int32_t dtype;         /* moe_dtype of every array but the codes' scales     */
  int32_t rows_per_gate; /* token t meets gate row t / rows_per_gate: 1 a gate
                            for each token, T one for all                      */
  float eps;             /* added to the mean square                           */
  float res_scale;       /* of the residual                                    */
} moe_norm_shape;

/* A matrix [T, d_model] of rows `ld` elements apart, ld >= d_model and
 * < 2^24; a null p with any ld is absent. */
typedef struct {
  void* p;
  int64_t ld;
} moe_rows;

typedef struct {
  moe_rows x;         /* in:  the residual, or absent                          */
  moe_rows y;         /* in:  the block's output, or absent                    */
  const void* w_post; /* [d_model] weights of the norm on y, or NULL: no norm  */
  const void* gate;   /* [ceil(T / rows_per_gate), d_model], or NULL: 1        */
  const void* w_pre;  /* [d_model] weights of the norm on r, or NULL: no h     */
  moe_rows r;         /* out: the new residual; absent where y is              */
  moe_rows h;         /* out: the next block's input; may be absent if q is not*/
  int8_t* q;          /* out: h's 8-bit codes [T, d_model] contiguous, or NULL */
  float* q_scale;     /* out: [T] their scales                                 */
} moe_norm_io;

/* moe_norm_residual -- the step between two blocks:
 *   r = res_scale x + gate (y rstd(y) w_post)
 *   h = r rstd(r) w_pre,  rstd(v) = 1 / sqrt(mean(v^2) + eps)
 * in fp32; r is rounded to dtype and h is the norm of the rounded r.  Absent
 * parts fall out: without y the call is the norm before the first block, h =
 * x rstd(x) w_pre (x needed, res_scale 1, w_post, gate and r absent); without
 * x the residual term is missing.  The sums of squares are fp32: they overflow
 * in rows of values beyond some 1e19 / sqrt(d_model), and with eps 0 a row of
 * zeros, or of values below some 1e-19, has no rstd.  q and q_scale are moe_quantize_rows of h.
 * r may be x itself (same p and ld).  16-byte aligned arrays, any strides. */
int moe_norm_residual(const moe_norm_shape* shape, const moe_norm_io* io, void* stream);

typedef struct {
  moe_rows r;         /* the forward pass's r (x where y is absent); needed
                         with w_pre                                            */
  moe_rows y;         /* the block's output, or absent                         */
  const void* w_post; /* as in the forward pass                                */
  const void* gate;
  const void* w_pre;
  moe_rows dr;        /* gradient at r, or absent: 0                           */
  moe_rows dh;        /* gradient at h; present with w_pre, and only then      */
  moe_rows dx;        /* out: gradient at x, or absent                         */
  moe_rows dy;        /* out: gradient at y; present with y, and only then     */
  void* dgate;        /* out: as gate, or NULL                                 */
  void* dw_post;      /* out: [d_model], or NULL                               */
  void* dw_pre;       /* out: [d_model], or NULL                               */
  int32_t accumulate; /* nonzero: dgate, dw_post and dw_pre are added to       */
  int32_t reserved;   /* 0                                                     */
} moe_norm_grad_io;

/* Bytes of `ws` that moe_norm_residual_backward needs for `shape` on the
 * current device; 0 if the shape is invalid. */
size_t moe_norm_residual_backward_workspace_bytes(const moe_norm_shape* shape);

/* moe_norm_residual_backward -- with the norms' values recomputed from r and y
 *   g  = dr + rstd(r) (dh w_pre - r rstd(r)^2 mean(dh w_pre r))
 *   dx = res_scale g
 *   dw_pre = sum_t dh r rstd(r)
 *   n  = y rstd(y);  dgate = sum over its tokens of g n w_post
 *   dw_post = sum_t g gate n,  c = g gate w_post
 *   dy = rstd(y) (c - n mean(c n))       (without w_post: n = y, dy = g gate)
 * in fp32, rounded once; the rounding of r in the forward pass is passed over.
 * A gradient whose forward value was absent must be absent.  dx and dy may each
 * be one of r, y, dr and dh themselves (same p and ld).  With T = 0 the vectors' gradients are
 * zeros (or stay, accumulating).  16-byte aligned arrays, any strides. */
int moe_norm_residual_backward(const moe_norm_shape* shape, const moe_norm_grad_io* io, void* ws,
                               void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_BLOCK_H */
