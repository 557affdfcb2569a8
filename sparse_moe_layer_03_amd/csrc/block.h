// Internal host-side interface of the kernels behind moe_block.h.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_block.h"
#include "train.h"

namespace moe {

// The arrays of a call.  A written one must not overlap any other, but for
// pairs that may be one and the same memory: rows of the same kind at the same
// start and stride, each element read before it is written, by one thread.
struct Arrays {
  struct Span {
    uintptr_t from, to;
    size_t step, width;  // bytes between rows and of a row; 0: one piece
    bool written, may_alias;
  };
  Span s[24];
  int n = 0;
  void add(const void* p, size_t bytes, bool written) {
    if (p == nullptr || bytes == 0) return;
    s[n++] = Span{(uintptr_t)p, (uintptr_t)p + bytes, 0, 0, written, false};
  }
  void rows(const void* p, int64_t ld, int M, int width, int size, bool written, bool may_alias) {
    if (p == nullptr || M == 0) return;
    const size_t step = (size_t)ld * size, wide = (size_t)width * size;
    s[n++] = Span{(uintptr_t)p, (uintptr_t)p + (size_t)(M - 1) * step + wide, step, wide, written, may_alias};
  }
  static bool apart(const Span& a, const Span& b) {
    if (a.from >= b.to || b.from >= a.to) return true;
    // columns of one wider matrix
    if (a.step == 0 || a.step != b.step) return false;
    const Span &lo = a.from <= b.from ? a : b, &hi = a.from <= b.from ? b : a;
    const size_t at = (hi.from - lo.from) % a.step;
    return at >= lo.width && at + hi.width <= a.step;
  }
  int check() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < i; ++j) {
        if ((!s[i].written && !s[j].written) || apart(s[i], s[j])) continue;
        // an output in an input's place
        if (s[i].written != s[j].written && s[i].may_alias && s[j].may_alias &&
            s[i].from == s[j].from && s[i].step == s[j].step)
          continue;
        return MOE_EINVAL;
      }
    return MOE_OK;
  }
};

// ---- selection (select.hip)

struct SelectArgs {
  const float* logits;
  int64_t ld;
  const float* bias;  // may be null
  int32_t* idx;
  float* gate;
  float scaling, eps;
  int T, E, k;
  int score, n_groups, top_groups, group_best, renorm;
};
int launch_select(const SelectArgs& a, hipStream_t st);

// Sums the K-split partial logits in split order, adds col_bias (nullable).
int launch_logits(const float* partials, int nsplit, const float* col_bias, int T, int E,
                  float* logits, hipStream_t st);
// The router's product (api.hip): logits [T, E], ws as moe_route's.
int run_router_logits(const moe_shape* s, const void* x, const void* w_router,
                      const float* logit_bias, float* logits, void* ws, hipStream_t st);

// moe_layer_backward, with another selection rule where `select` is given
// (train_api.hip).
int run_layer_backward(const moe_shape* s, const moe_select_params* select,
                       const moe_backward_io* io, void* ws, hipStream_t st);

// The gradient at the logits; `dl` as in TokenArgs (ep elements a row, halves
// of them), either of dlogits and dl may be null.
struct SelectBwdArgs {
  const float* logits;
  int64_t ld;
  const int32_t* idx;
  const float* dgate;
  float* dlogits;
  void* dl;
  float scaling, eps;
  int T, E, k;
  int score, renorm;
  int ep, halves;
  int32_t* route_offs;  // with dl: 0, T and the bounds of nsplit token ranges,
  int32_t* split_offs;  // as in TokenArgs
  int nsplit;
};
int launch_select_bwd(const SelectBwdArgs& a, hipStream_t st);

// ---- 8-bit rows and products (quant.hip, gmm_i8.hip, i8_general.hip)

// Quantises the rows of x; the rows' codes of a bf16 or fp32 array.
int launch_quantize(int dtype, const void* x, int64_t ldx, int M, int K, int8_t* q, int64_t ldq,
                    float* scale, const int32_t* m_used, hipStream_t st);

// The FFN rows, sorted by expert: for p < offsets[n_ffn], the token perm[p] / k
// and its scale.
int launch_row_tokens(const float* xs, const int32_t* perm, const int32_t* offsets, int n_ffn, int Tk,
                      int k, int32_t* tok, float* row_scale, hipStream_t st);

// out[p, j] = (sum_r a[p, r] b_e[j, r]) sa[p] sb[e, j]; with b2, SwiGLU of the
// products by b (gate) and b2 (up), a's row for p being tok[p].
struct I8Args {
  const int8_t* a;
  const float* sa;
  const int8_t *b, *b2;
  const float *sb, *sb2;
  const int32_t* tok;      // with b2
  uint32_t a_bytes;        // of a, with b2: less than 2^31 - 2^16
  void* out;
  const int32_t* offsets;  // may be null with one group
  int64_t lda, ldo;
  int ngroups, M, N, K;
  int rows;                // about as many of the M are in use
  int nsplit;              // ranges of the reduction, their sums in `part`
  int32_t* part;           // [nsplit, M, N]
};
bool i8_mfma_ok(int N, int K, int64_t lda, int64_t ldo);
int launch_i8_mfma(int out_dtype, const I8Args& g, hipStream_t st);
int launch_i8_general(int out_dtype, const I8Args& g, hipStream_t st);
int launch_i8_join(int out_dtype, const I8Args& g, hipStream_t st);

// ---- norms (norm.hip)

int launch_norm(const moe_norm_shape& s, const moe_norm_io& io, hipStream_t st);
// Workgroups of the backward pass, and so rows of its partial sums.
int norm_bwd_groups(int T, int d, int cus);
size_t norm_bwd_ws_bytes(const moe_norm_shape& s, int cus);
int launch_norm_bwd(const moe_norm_shape& s, const moe_norm_grad_io& io, void* ws, int cus,
                    hipStream_t st);

// as the accessors of internal.h
unsigned check_word_select(bool clear);
unsigned check_word_quant(bool clear);
unsigned check_word_gmm_i8(bool clear);
unsigned check_word_i8_general(bool clear);

}  // namespace moe
