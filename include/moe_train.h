/*
 * moe_train.h -- C ABI of the MI355X (gfx950) sparse MoE layer's training
 * operators: the matrix products grouped by expert in the three forms that
 * training needs, the layer's backward pass, and an AdamW step over many
 * tensors.  Same library, status codes, types and layer shape as moe.h.
 *
 * Conventions (as in moe.h, with what differs stated at each call)
 *   - Pointers to arrays are DEVICE pointers owned by the caller; scratch
 *     comes from `ws`.  The library allocates, frees and keeps nothing after
 *     the call returns.  `stream` is a hipStream_t of the current device
 *     (NULL = the default stream); calls only enqueue work and can be
 *     captured into a HIP graph.  A workspace serves one call at a time: two
 *     calls, or two graphs, that may overlap need one each.
 *   - Return value: MOE_OK (0) or a negative moe_status.  Arguments are
 *     checked on the host before anything is enqueued.  Offsets and routing
 *     arrays in device memory cannot be: the kernels keep every row that they
 *     name inside the arrays, so wrong ones give wrong values and never an
 *     access out of range (the debug build reports them, moe_debug_checks).
 *   - Sums are formed in a fixed order, without atomics: the same call gives
 *     the same bits.
 */
#ifndef MOE_MI355X_TRAIN_H
#define MOE_MI355X_TRAIN_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The three products of a grouped linear map c = a W_e^T, e the group that
 * owns the row: rows offsets[e] <= p < offsets[e+1]. */
typedef enum {
  MOE_GMM_FWD = 0, /* c[p, :]  = a[p, :] W_e^T                             */
  MOE_GMM_DX = 1,  /* a[p, :]  = c[p, :] W_e        (gradient of the rows) */
  MOE_GMM_DW = 2   /* W_e      = sum_p c[p, :]^T a[p, :]  (of the weights) */
} moe_gmm_form;

/* Sizes of one grouped product.
 *   a [M, K] with lda elements from row to row, c [M, N] with ldc,
 *   W [n_groups, N, K] contiguous.
 * Limits: 1 <= n_groups <= 1024; 0 <= M < 2^27; 1 <= N, K <= 2^20;
 * K <= lda < 2^24; N <= ldc < 2^24.  Any sizes and strides within them; rows
 * and strides that are multiples of 16 bytes take the fast kernels. */
typedef struct {
  int32_t form;       /* moe_gmm_form                                      */
  int32_t dtype;      /* moe_dtype of the two arrays that are read         */
  int32_t out_dtype;  /* of the array that is written: dtype or MOE_F32    */
  int32_t accumulate; /* nonzero: add to what the written array holds      */
  int32_t n_groups;   /* experts                                           */
  int32_t M;          /* rows that a and c have room for; the tiles go by
                         it, so the rows in use where the host knows them  */
  int32_t N, K;       /* output and input width of the map                 */
  int64_t lda, ldc;   /* elements between rows of a and of c               */
} moe_gmm_shape;

/* Bytes of `ws` that moe_grouped_matmul needs for `shape` on the current
 * device (partial sums of products whose reduction is split to fill the
 * chip; 0 for most shapes, then ws may be NULL).  0 too if the shape is
 * invalid. */
size_t moe_grouped_matmul_workspace_bytes(const moe_gmm_shape* shape);

/* moe_grouped_matmul -- one of the three products above.
 *   FWD: lhs = a, rhs = W, out = c;  DX: lhs = c, rhs = W, out = a;
 *   DW:  lhs = c, rhs = a, out = W.
 *   offsets [n_groups + 1] int32, ascending: from moe_dispatch (its first
 *   n_ffn + 1 entries).  A group may be empty; rows behind offsets[n_groups]
 *   are neither read nor written.  DW writes every group: zeros where a
 *   group is empty (unless it accumulates).
 * Products are summed in fp32 and rounded once to out_dtype (an accumulated
 * value is added in fp32 before that).  out must not overlap lhs or rhs.
 * Pointers aligned to 16 bytes (offsets 4); lhs and the rows of rhs may be
 * NULL when M = 0. */
int moe_grouped_matmul(const moe_gmm_shape* shape, const int32_t* offsets, const void* lhs,
                       const void* rhs, void* out, void* ws, void* stream);

/* Arrays of the layer's backward pass (a host struct of device pointers,
 * read during the call).  E = n_ffn + n_zero. */
typedef struct {
  /* what the forward pass had and left */
  const void* x;             /* [T, d_model] dtype                              */
  const void* w_router;      /* [E, d_model] dtype                              */
  const float* logits;       /* [T, E] fp32: moe_route's logits_out             */
  const int32_t* topk_idx;   /* [T, top_k]                                      */
  const float* topk_gate;    /* [T, top_k] fp32                                 */
  const int32_t* offsets;    /* [E + 1]                                         */
  const int32_t* perm;       /* [T * top_k]                                     */
  const int32_t* inv_perm;   /* [T * top_k]                                     */
  const void* w_gate;        /* [n_ffn, d_ff, d_model] dtype                    */
  const void* w_up;          /* [n_ffn, d_ff, d_model] dtype                    */
  const void* w_down;        /* [n_ffn, d_model, d_ff] dtype                    */
  const void* dy;            /* [T, d_model] dtype: gradient at y               */
  /* gradients */
  void* dx;                  /* [T, d_model] dtype                              */
  float* dgate;              /* [T, top_k] fp32: gradient at topk_gate          */
  float* dlogits;            /* [T, E] fp32, or NULL                            */
  void* dw_router;           /* [E, d_model] dtype, or NULL                     */
  void* dw_gate;             /* [n_ffn, d_ff, d_model] dtype                    */
  void* dw_up;               /* [n_ffn, d_ff, d_model] dtype                    */
  void* dw_down;             /* [n_ffn, d_model, d_ff] dtype                    */
  int32_t accumulate;        /* nonzero: weight gradients are added to what is there */
  int32_t reserved;          /* 0                                               */
} moe_backward_io;

/* Bytes of `ws` that moe_layer_backward needs for `shape` on the current
 * device; 0 if the shape is invalid. */
size_t moe_layer_backward_workspace_bytes(const moe_shape* shape);

/* moe_layer_backward -- gradients of one layer pass (moe_route,
 * moe_dispatch, moe_expert_ffn, moe_combine) from the gradient dy at y.
 * H is computed again from x, so nothing of the experts' inner values has to
 * be kept:
 *   z = x Wg^T, u = x Wu^T, h = silu(z) u, dh = dy Wd          (per FFN row)
 *   dgate[t,j] = <dh, h> for an FFN expert, <dy[t], x[t]> for an identity one
 *   dz = gate dh u silu'(z),  du = gate dh silu(z)
 *   dw_gate = dz^T x,  dw_up = du^T x,  dw_down = dy^T (gate h)
 *   dlogits = p (dp - sum_e p dp),  p = softmax(logits),
 *             dp[t, e] = routed_scaling sum_{j: topk_idx[t,j] = e} dgate[t,j]
 *   dw_router = dlogits^T x
 *   dx[t] = sum_{FFN j} (dz Wg + du Wu) + (sum_{identity j} gate) dy[t]
 *           + dlogits[t] w_router
 * The selection itself and the bias that steers it have no gradient; a
 * selection that moe_route did not make may name an expert twice.
 * moe_route's logit_bias enters p as the logits do: its gradient is
 * sum_t dlogits[t, :], which is left to the caller to form.  With
 * logits NULL the router is left out: w_router, dlogits and dw_router must
 * be NULL then, and dx holds the experts' part alone.  In bf16, dz, du and
 * gate h are rounded to bf16 where they enter a product, and dlogits enters
 * as two bf16 values, the rounded one and what the rounding leaves; all else
 * is fp32 until the results are rounded.  With `accumulate` the old value is
 * added in fp32 and the sum rounded to dtype: a bf16 gradient that is summed
 * over many passes is rounded in each of them.
 * Shape limits as in moe.h, and T * top_k < 2^27, d_model <= 2^20, d_ff <=
 * 2^19; outputs must not overlap inputs or each other. */
int moe_layer_backward(const moe_shape* shape, const moe_backward_io* io, void* ws, void* stream);

/* Hyper-parameters of an AdamW step (host struct, copied into the launch);
 * finite in fp32. */
typedef struct {
  double lr;           /* learning rate, >= 0                                */
  double beta1, beta2; /* decay of the moments, in [0, 1)                    */
  double eps;          /* >= 1e-30                                           */
  int32_t state_bits;  /* 32: fp32 moments; 8: e4m3 codes with block scales  */
  uint32_t seed;       /* of the 8-bit states' random rounding               */
} moe_adamw_params;

/* One parameter tensor (host struct of device pointers).  Arrays are
 * contiguous with n elements, n >= 0; all pointers 16-byte aligned. */
typedef struct {
  void* param;          /* updated in place                                  */
  const void* grad;
  float* master;        /* fp32 copy that is updated, param being its
                           rounding; NULL: param itself is the value; an
                           fp32 param may be its own                         */
  void* m;              /* first moment: fp32 [n], or e4m3 codes [n]         */
  void* v;              /* second moment: fp32 [n], or e4m3 codes of its root*/
  float* m_scale;       /* 8-bit states: fp32 [ceil(n / 256)], else NULL     */
  float* v_scale;
  int64_t n;
  int32_t param_dtype;  /* moe_dtype                                         */
  int32_t grad_dtype;   /* moe_dtype                                         */
  double weight_decay;  /* >= 0, finite in fp32                              */
} moe_adamw_tensor;

/* Memory of the optimizer; lives in DEVICE memory, caller-owned,
 * zero-initialised before the first step, 16-byte aligned.  The step count
 * is kept here so that a captured graph counts its replays. */
typedef struct {
  int32_t step;      /* steps taken                                          */
  int32_t skipped;   /* steps skipped for a non-finite grad_scale            */
  uint32_t arrived;  /* used within a call, 0 between calls                  */
  int32_t reserved;
} moe_adamw_state;

/* moe_adamw -- one AdamW step over n_tensors tensors (host array, read
 * during the call), 48 of them in a launch:
 *   t = step + 1;  g = grad_scale * grad
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr (m / (1 - beta1^t)) / (sqrt(v / (1 - beta2^t)) + eps)
 * in fp32.  grad_scale (device, one fp32, or NULL for 1): a clipping factor
 * or an inverse loss scale computed on the device; when it is not finite
 * nothing changes but `skipped`.  lr_scale (device, one fp32, or NULL for
 * 1) multiplies lr, for a schedule under graph replay; it is not checked, and
 * one that is not finite reaches every parameter.
 * 8-bit states: elements 256 b .. 256 b + 255 share a scale, the block's
 * largest magnitude / 448; element i stands for code * scale, for v the
 * square of that.  The new value is rounded at random to one of the two
 * neighbouring codes so that its mean (the mean of its square, for v) is
 * kept, to 2^-16 of the codes' distance: rounding to nearest would hold on to
 * an average that moves by less than half a code each step.  A v > 0 never
 * becomes 0.  The random numbers depend on (seed, step, tensor's place in the
 * list, i) only.  A gradient
 * that is not finite reaches its own element (8 bits: its block); to leave a
 * step out, pass a grad_scale that is not finite.  An array that is written
 * must not overlap any other of the list (a tied weight is listed once). */
int moe_adamw(const moe_adamw_params* params, const moe_adamw_tensor* tensors, int32_t n_tensors,
              moe_adamw_state* state, const float* grad_scale, const float* lr_scale,
              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MI355X_TRAIN_H */
