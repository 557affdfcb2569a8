// Internal host-side interface of the training operators' kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe_train.h"
#include "internal.h"

namespace moe {

// Rows of a product: row tiles are counted in 22 bits, and the scan over the
// groups' tiles stays inside an int whatever the offsets hold.
constexpr int kGmmMaxRows = 1 << 27;

// Grouped products in the kernels' terms: out[i, j] = sum_r A(i, r) B(j, r)
// for every group.  FWD and DX: i runs over the group's rows, r over R.  DW:
// r runs over the group's rows, i over I.  j runs over J.  Up to three
// products over the same groups share a launch (FWD: with the same a; DX:
// one only).
struct GmmSub {
  const void* a;
  const void* b;
  void* out;
  int64_t lda, ldb, ldo;   // elements between rows of the arrays
  int I, J;
};
struct GmmArgs {
  GmmSub s[3];
  int nsub;
  int ngroups;
  const int32_t* offsets;  // [ngroups + 1]
  int M;                   // rows that the row arrays hold
  int R;                   // FWD, DX: length of the reduction
  int RB;                  // DX: rows that a group of b, and of b2, holds; behind
                           // them the reduction reads zeros
  int r_switch;            // DX: reduction rows from here on (a multiple of 64)
                           // come from b2, from its first one (0: none; bf16:
                           // on the MFMA kernels' 16-byte rows only)
  const void* b2;          // DX: see r_switch; SwiGLU step: w_up
  int64_t b_group;         // elements between groups of b (FWD, DX)
  int64_t out_group;       // elements between groups of out (DW)
  float* part;             // split reductions: fp32 partial outputs, split-major
  int64_t part_stride;     // elements between splits in `part`
  int nsplit;              // ranges of the reduction (> 1: one product only)
  int accumulate;
  // SwiGLU's backward step (FWD): z = a b^T, u = a b2^T
  const float* gate;       // per row
  const float* dh;         // [rows, J] fp32
  void* dzu;               // [rows, 2 J]
  void* hs;                // [rows, J]
  float* dpart;            // [rows, swiglu_parts()]
};

// Any sizes, strides and element types.
int launch_gmm_general(int form, int dtype, int out_dtype, const GmmArgs& g, hipStream_t st);
// bf16 products on bf16 MFMAs (gmm_mfma.hip; FWD: one product).
// Whether a product can run there: 16-byte rows and row starts, and sizes
// that 32-bit offsets within a tile reach.
bool mfma_ok(int form, int dtype, int N, int K, int64_t lda, int64_t ldc);
int launch_gmm_mfma(int form, int out_dtype, const GmmArgs& g, hipStream_t st);
int launch_swiglu_mfma(const GmmArgs& g, hipStream_t st);
int swiglu_parts(int M, int ngroups, int f);  // partial sums of dgate per row

// Sums `part` into out (rounded, added to when accumulating).
int launch_gmm_join(int form, int out_dtype, const GmmArgs& g, hipStream_t st);

// The layer's shape checks (moe.h's limits).
int check_shape(const moe_shape* s);

int launch_adamw(const moe_adamw_params* hp, const moe_adamw_tensor* tensors, int n_tensors,
                 moe_adamw_state* state, const float* grad_scale, const float* lr_scale,
                 hipStream_t st);
uint64_t adamw_max_elements();

// as the accessors of internal.h
unsigned check_word_gmm_general(bool clear);
unsigned check_word_gmm_mfma(bool clear);
unsigned check_word_layer_bwd(bool clear);

// ---- the layer's backward pass beside its products

// The FFN rows of x and dy grouped by expert, and their gates: for p <
// offsets[n_ffn], row perm[p] / k of each, gate_rows[p] = gate[perm[p]].
int launch_gather2(int dtype, const void* x, const void* dy, const float* gate, const int32_t* perm,
                   const int32_t* offsets, int n_ffn, int Tk, int k, int d, void* xp, void* dyp,
                   float* gate_rows, hipStream_t st);

// fp32 layers.  Per FFN row p: h, dz, du from z, u and dh ([rows, f], z and u
// in `zu` [rows, 2 f]), the row's gate applied; dzu [rows, 2 f], hs [rows, f],
// dgate_part[p] = <dh, h>.
int launch_swiglu_bwd(const float* zu, const float* dh, const float* gate_rows,
                      const int32_t* offsets, int n_ffn, int Tk, int f, float* dzu, float* hs,
                      float* dgate_part, hipStream_t st);

// Per token: dgate (parts: partial sums per FFN row), then, with logits,
// dlogits (fp32 if not null), its operand `dl` of the router's products, and
// their row bounds: route_offs[0..1] = 0, T and split_offs[s] = s * T / nsplit.
// dl in fp32: rows of ep elements, zeros behind E.  In bf16 rows of 2 ep: the
// rounded values and, ep behind, what the rounding left of them.
struct TokenArgs {
  const void* x;
  const void* dy;
  const float* logits;
  const int32_t* idx;
  const int32_t* inv_perm;
  const float* part;
  float* dgate;
  float* dlogits;
  void* dl;
  int32_t* route_offs;
  int32_t* split_offs;
  float scaling;
  int T, d, E, k, n_ffn, parts, ep, nsplit;
};
int launch_token_bwd(int dtype, const TokenArgs& a, hipStream_t st);

// dx[t] = sum over FFN slots of dx_rows + (identity gates) dy[t] + dxr[t]
// (both fp32; dxr may be null), rounded once.
int launch_dx(int dtype, const float* dx_rows, const void* dy, const float* dxr, const int32_t* idx,
              const float* gate, const int32_t* inv_perm, int T, int d, int k, int n_ffn, void* dx,
              hipStream_t st);

}  // namespace moe
