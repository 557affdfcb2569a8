// C ABI of the training operators: argument checks, workspace layout and the
// launch sequence of each call.  Every check runs on the host before any
// work is enqueued; no call allocates, frees or synchronises.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "common.h"
#include "train.h"

namespace moe {

static bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
static long cdiv(long a, long b) { return (a + b - 1) / b; }
static int elem_size(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }

static int check_gmm(const moe_gmm_shape* s) {
  if (s == nullptr) return MOE_EINVAL;
  if (s->form < MOE_GMM_FWD || s->form > MOE_GMM_DW || s->n_groups < 1 || s->M < 0 || s->N < 1 ||
      s->K < 1 || s->lda < s->K || s->ldc < s->N)
    return MOE_EINVAL;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) return MOE_EUNSUPPORTED;
  if (s->out_dtype != s->dtype && s->out_dtype != MOE_F32) return MOE_EUNSUPPORTED;
  if (s->n_groups > 1024 || s->M >= kGmmMaxRows || s->N > (1 << 20) || s->K > (1 << 20) || s->lda >= (1 << 24) ||
      s->ldc >= (1 << 24))
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// A product with too few output tiles to fill the chip has its reduction cut
// into this many ranges, each at least 256 long, whose fp32 partial outputs
// are joined by a second kernel.  A function of the sizes and the device's CU
// count only: it sizes the workspace (at most `fill` tiles per CU: 16 MiB each).
static int gmm_nsplit(int form, long G, long M, long I, long J, long R, int fill, int cus) {
  const long jt = cdiv(J, 128);
  const long tiles = form == MOE_GMM_DW ? G * cdiv(I, 128) * jt : (M / 128 + std::min(G, M)) * jt;
  const long red = form == MOE_GMM_DW ? M / G : R;
  if (tiles < 1) return 1;
  return (int)std::max(1l, std::min({64l, (long)fill * cus / tiles, red / 256}));
}

static int gmm_splits_of(const moe_gmm_shape* s, int cus) {
  const bool fwd = s->form == MOE_GMM_FWD;
  // fp32 MFMAs are busy with two workgroups on a CU
  const int fill = s->dtype == MOE_F32 ? 2 : 1;
  return gmm_nsplit(s->form, s->n_groups, s->M, s->N, fwd ? s->N : s->K, fwd ? s->K : s->N, fill, cus);
}

static size_t gmm_part_bytes(const moe_gmm_shape* s, int nsplit) {
  if (nsplit <= 1) return 0;
  const size_t out = s->form == MOE_GMM_DW ? (size_t)s->n_groups * s->N * s->K
                                           : (size_t)s->M * (s->form == MOE_GMM_FWD ? s->N : s->K);
  return up256(out * nsplit * sizeof(float));
}

// Runs products, a split reduction joined.
static int run_gmm(int form, int dtype, int out_dtype, const GmmArgs& g, hipStream_t st) {
  const bool fwd = form == MOE_GMM_FWD, dx = form == MOE_GMM_DX;
  bool mfma = !(fwd && g.nsub > 1);
  for (int q = 0; q < g.nsub; ++q) {
    const GmmSub& s = g.s[q];
    const int64_t lda = dx ? s.ldo : fwd ? s.lda : s.ldb, ldc = fwd ? s.ldo : s.lda;
    const int N = fwd ? s.J : dx ? g.R : s.I, K = fwd ? g.R : s.J;
    mfma = mfma && al16(s.a) && al16(s.b) && al16(s.out) && mfma_ok(form, dtype, N, K, lda, ldc);
  }
  const int rc = mfma ? launch_gmm_mfma(form, out_dtype, g, st)
                      : launch_gmm_general(form, dtype, out_dtype, g, st);
  if (rc || g.nsplit <= 1) return rc;
  return launch_gmm_join(form, out_dtype, g, st);
}

// ---- the layer's backward pass: workspace

constexpr int kRouteSplits = 16;  // most token ranges of the router's weight gradient

struct BwdLayout {
  size_t xp, dyp, gates, zu, dh, dzu, hs, part, dl, offs, dxr, drp, total;
  int ep, halves, nsplit, parts;
};

static BwdLayout bwd_layout(const moe_shape* s) {
  const size_t es = elem_size(s->dtype);
  const size_t E = (size_t)s->n_ffn + s->n_zero, rows = (size_t)s->T * s->top_k;
  const size_t d = s->d_model, f = s->d_ff;
  BwdLayout w;
  // In bf16 dlogits enters the router's products as two bf16 values, the
  // rounded one and the rest: scores and gates are fp32 in this layer, and so
  // stay their gradients.  64: where the second part begins, a step's start.
  w.halves = s->dtype == MOE_BF16 ? 2 : 1;
  w.ep = (int)((E + 63) & ~(size_t)63);
  // the router's weight gradient has few tiles and a reduction over all
  // tokens: as many ranges of at least 256 of them as give every CU a tile
  const int cus = device_cu_count();
  w.nsplit = (int)std::max(1l, std::min({(long)kRouteSplits, (long)s->T / 256,
                                         (cus > 0 ? cus : 256) /
                                             (cdiv(w.ep * w.halves, 256) * cdiv(d, 256))}));
  w.parts = s->dtype == MOE_BF16 ? swiglu_parts((int)rows, s->n_ffn, s->d_ff) : 1;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up256(off + bytes);
    return at;
  };
  w.xp = take(rows * d * es);   // with dyp behind it, later the rows' gradients:
  w.dyp = take(rows * d * es);  // fp32 [rows, d]
  w.gates = take(rows * 4);
  w.zu = take(s->dtype == MOE_BF16 ? 0 : rows * 2 * f * 4);
  w.dh = take(rows * f * 4);
  w.dzu = take(rows * 2 * f * es);
  w.hs = take(rows * f * es);
  w.part = take(rows * w.parts * 4);
  w.dl = take((size_t)s->T * w.ep * w.halves * es);
  w.offs = take((2 + kRouteSplits + 1) * sizeof(int32_t));
  w.dxr = take((size_t)s->T * d * 4);
  w.drp = take((size_t)w.ep * w.halves * d * 4 * w.nsplit);
  w.total = off;
  return w;
}

static int check_backward_shape(const moe_shape* s) {
  const int rc = check_shape(s);
  if (rc) return rc;
  // (2 d_ff and d_model are row lengths of the products)
  return (long)s->T * s->top_k < kGmmMaxRows && s->d_model <= (1 << 20) && s->d_ff <= (1 << 19)
             ? MOE_OK
             : MOE_EUNSUPPORTED;
}

static int check_backward(const moe_shape* s, const moe_backward_io* io) {
  const int rc = check_backward_shape(s);
  if (rc) return rc;
  if (!io) return MOE_EINVAL;
  if (!io->x || !io->topk_idx || !io->topk_gate || !io->offsets || !io->perm || !io->inv_perm ||
      !io->w_gate || !io->w_up || !io->w_down || !io->dy || !io->dx || !io->dgate ||
      !io->dw_gate || !io->dw_up || !io->dw_down || io->reserved != 0)
    return MOE_EINVAL;
  if (io->logits ? (!io->w_router || !io->dw_router)
                 : (io->w_router || io->dw_router || io->dlogits))
    return MOE_EINVAL;
  if (!al16(io->x) || !al16(io->w_router) || !al16(io->w_gate) || !al16(io->w_up) ||
      !al16(io->w_down) || !al16(io->dy) || !al16(io->dx) || !al16(io->dw_router) ||
      !al16(io->dw_gate) || !al16(io->dw_up) || !al16(io->dw_down) || !al4(io->logits) ||
      !al4(io->topk_idx) || !al4(io->topk_gate) || !al4(io->offsets) || !al4(io->perm) ||
      !al4(io->inv_perm) || !al4(io->dgate) || !al4(io->dlogits))
    return MOE_EALIGN;
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grouped_matmul_workspace_bytes(const moe_gmm_shape* s) {
  if (check_gmm(s) != MOE_OK) return 0;
  const int cus = device_cu_count();
  return cus > 0 ? gmm_part_bytes(s, gmm_splits_of(s, cus)) : 0;
}

int moe_grouped_matmul(const moe_gmm_shape* s, const int32_t* offsets, const void* lhs,
                       const void* rhs, void* out, void* ws, void* stream) {
  const int rc = check_gmm(s);
  if (rc) return rc;
  const bool dw = s->form == MOE_GMM_DW;
  // with no rows, arrays that have one row per token may be null
  const bool none = s->M == 0;
  if (!offsets || (!lhs && !none) || (!rhs && !(none && dw)) || (!out && !(none && !dw)))
    return MOE_EINVAL;
  if (!al4(offsets) || !al16(lhs) || !al16(rhs) || !al16(out) || !al16(ws)) return MOE_EALIGN;
  const int cus = device_cu_count();
  if (cus <= 0) return MOE_EHIP;
  GmmArgs g{};
  g.nsub = 1;
  g.offsets = offsets;
  g.ngroups = s->n_groups;
  g.M = s->M;
  g.b_group = g.out_group = (int64_t)s->N * s->K;
  g.accumulate = s->accumulate != 0;
  g.nsplit = gmm_splits_of(s, cus);
  if (g.nsplit > 1 && !ws) return MOE_EINVAL;
  g.part = (float*)ws;
  GmmSub& p = g.s[0];
  p.a = lhs;
  p.b = rhs;
  p.out = out;
  p.I = s->N;
  if (s->form == MOE_GMM_FWD) {
    p.lda = s->lda;
    p.ldb = s->K;
    p.ldo = s->ldc;
    p.J = s->N;
    g.R = s->K;
    g.part_stride = (int64_t)s->M * s->N;
  } else if (s->form == MOE_GMM_DX) {
    p.lda = s->ldc;
    p.ldb = s->K;
    p.ldo = s->lda;
    p.J = s->K;
    g.R = s->N;
    g.part_stride = (int64_t)s->M * s->K;
  } else {
    p.lda = s->ldc;
    p.ldb = s->lda;
    p.ldo = s->K;
    p.J = s->K;
    g.part_stride = (int64_t)s->n_groups * s->N * s->K;
  }
  g.RB = g.R;
  if (none && !dw) return MOE_OK;
  return run_gmm(s->form, s->dtype, s->out_dtype, g, (hipStream_t)stream);
}

size_t moe_layer_backward_workspace_bytes(const moe_shape* s) {
  if (check_backward_shape(s) != MOE_OK) return 0;
  return bwd_layout(s).total;
}

int moe_layer_backward(const moe_shape* s, const moe_backward_io* io, void* ws, void* stream) {
  int rc = check_backward(s, io);
  if (rc) return rc;
  if (!ws) return MOE_EINVAL;
  if (!al16(ws)) return MOE_EALIGN;
  hipStream_t st = (hipStream_t)stream;
  const BwdLayout w = bwd_layout(s);
  char* base = (char*)ws;
  const int E = s->n_ffn + s->n_zero, Tk = s->T * s->top_k;
  const int d = s->d_model, f = s->d_ff, dt = s->dtype, es = elem_size(dt);
  char *xp = base + w.xp, *dyp = base + w.dyp, *dzu = base + w.dzu, *hs = base + w.hs;
  float *zu = (float*)(base + w.zu), *dh = (float*)(base + w.dh), *part = (float*)(base + w.part);
  float *dxr = (float*)(base + w.dxr), *drp = (float*)(base + w.drp);
  char* dl = base + w.dl;
  int32_t *route_offs = (int32_t*)(base + w.offs), *split_offs = route_offs + 2;

  float* gates = (float*)(base + w.gates);
  const int acc = io->accumulate != 0;
  if ((rc = launch_gather2(dt, io->x, io->dy, io->topk_gate, io->perm, io->offsets, s->n_ffn, Tk,
                           s->top_k, d, xp, dyp, gates, st)))
    return rc;

  GmmArgs g{};
  g.offsets = io->offsets;
  g.ngroups = s->n_ffn;
  g.M = Tk;
  g.nsplit = 1;
  g.b_group = g.out_group = (int64_t)d * f;
  // the gradient at H, before the gate
  g.nsub = 1;
  g.s[0] = {dyp, io->w_down, dh, d, f, f, 0, f};
  g.R = g.RB = d;
  if ((rc = run_gmm(MOE_GMM_DX, dt, MOE_F32, g, st))) return rc;
  // z and u again, and SwiGLU's step (in bf16 behind the products' K loop)
  if (dt == MOE_BF16) {
    g.s[0] = {xp, io->w_gate, nullptr, d, d, 0, 0, f};
    g.b2 = io->w_up;
    g.gate = gates;
    g.dh = dh;
    g.dzu = dzu;
    g.hs = hs;
    g.dpart = part;
    if ((rc = launch_swiglu_mfma(g, st))) return rc;
  } else {
    g.nsub = 2;
    g.s[0] = {xp, io->w_gate, zu, d, d, 2 * f, 0, f};
    g.s[1] = {xp, io->w_up, zu + f, d, d, 2 * f, 0, f};
    if ((rc = run_gmm(MOE_GMM_FWD, dt, MOE_F32, g, st))) return rc;
    if ((rc = launch_swiglu_bwd(zu, dh, gates, io->offsets, s->n_ffn, Tk, f, (float*)dzu,
                                (float*)hs, part, st)))
      return rc;
  }
  // gradients of the experts' weights
  g.nsub = 3;
  g.s[0] = {dzu, xp, io->dw_gate, 2 * f, d, d, f, d};
  g.s[1] = {dzu + (size_t)f * es, xp, io->dw_up, 2 * f, d, d, f, d};
  g.s[2] = {dyp, hs, io->dw_down, d, f, f, d, f};
  g.accumulate = acc;
  if ((rc = run_gmm(MOE_GMM_DW, dt, dt, g, st))) return rc;
  // gradients of the rows, one reduction over gate's and up's columns, in fp32
  // (a bf16 rounding of each row would be a third of dx's error) over x's and
  // dy's rows, which are not needed any more
  float* dx_rows = (float*)xp;
  g.nsub = 1;
  g.s[0] = {dzu, io->w_gate, dx_rows, 2 * f, d, d, 0, d};
  g.b2 = io->w_up;
  g.R = 2 * f;
  g.RB = g.r_switch = f;
  g.accumulate = 0;
  if ((rc = run_gmm(MOE_GMM_DX, dt, MOE_F32, g, st))) return rc;

  // gradients at the gates and logits, and the router's products
  TokenArgs a{};
  a.x = io->x;
  a.dy = io->dy;
  a.logits = io->logits;
  a.idx = io->topk_idx;
  a.inv_perm = io->inv_perm;
  a.part = part;
  a.dgate = io->dgate;
  a.dlogits = io->dlogits;
  a.dl = dl;
  a.route_offs = route_offs;
  a.split_offs = split_offs;
  a.scaling = s->routed_scaling;
  a.T = s->T;
  a.d = d;
  a.E = E;
  a.k = s->top_k;
  a.n_ffn = s->n_ffn;
  a.parts = w.parts;
  a.ep = w.ep;
  a.nsplit = w.nsplit;
  if ((rc = launch_token_bwd(dt, a, st))) return rc;
  if (io->logits) {
    GmmArgs r{};
    r.nsub = 1;
    r.M = s->T;
    r.nsplit = 1;
    // dlogits W_router, fp32 (dlogits' rows have zeros behind E, where
    // w_router has none)
    const int wide = w.ep * w.halves;
    r.s[0] = {dl, io->w_router, dxr, wide, d, d, 0, d};
    r.offsets = route_offs;
    r.ngroups = 1;
    r.R = wide;
    r.RB = E;
    r.b2 = io->w_router;
    r.r_switch = w.halves == 2 ? w.ep : 0;
    if ((rc = run_gmm(MOE_GMM_DX, dt, MOE_F32, r, st))) return rc;
    // dlogits^T x over ranges of the tokens, both parts, then their sum
    r.s[0] = {dl, io->x, drp, wide, d, d, wide, d};
    r.out_group = (int64_t)wide * d;
    r.offsets = split_offs;
    r.ngroups = w.nsplit;
    if ((rc = run_gmm(MOE_GMM_DW, dt, MOE_F32, r, st))) return rc;
    r.part = drp;
    r.part_stride = (int64_t)w.ep * d;
    r.nsplit = w.nsplit * w.halves;
    r.ngroups = 1;
    r.s[0].out = io->dw_router;
    r.s[0].I = E;
    r.accumulate = acc;
    rc = launch_gmm_join(MOE_GMM_DW, dt, r, st);
    if (rc) return rc;
  }
  return launch_dx(dt, dx_rows, io->dy, io->logits ? dxr : nullptr, io->topk_idx, io->topk_gate,
                   io->inv_perm, s->T, d, s->top_k, s->n_ffn, io->dx, st);
}

int moe_adamw(const moe_adamw_params* hp, const moe_adamw_tensor* tensors, int32_t n_tensors,
              moe_adamw_state* state, const float* grad_scale, const float* lr_scale,
              void* stream) {
  if (!hp || !tensors || !state || n_tensors < 1) return MOE_EINVAL;
  // as the kernel takes them: fp32
  if (!isfinite((float)hp->lr) || !isfinite(hp->beta1) || !isfinite(hp->beta2) ||
      !isfinite((float)hp->eps))
    return MOE_ENONFINITE;
  if (hp->lr < 0 || hp->beta1 < 0 || hp->beta1 >= 1 || hp->beta2 < 0 || hp->beta2 >= 1 ||
      (float)hp->eps < 1e-30f)
    return MOE_EINVAL;
  if (hp->state_bits != 32 && hp->state_bits != 8) return MOE_EUNSUPPORTED;
  if (!al16(state) || !al4(grad_scale) || !al4(lr_scale)) return MOE_EALIGN;
  uint64_t n = 0;
  for (int k = 0; k < n_tensors; ++k) {
    const moe_adamw_tensor& t = tensors[k];
    if (t.n < 0) return MOE_EINVAL;
    if (!isfinite((float)t.weight_decay)) return MOE_ENONFINITE;
    if (t.weight_decay < 0) return MOE_EINVAL;
    if ((t.param_dtype != MOE_F32 && t.param_dtype != MOE_BF16) ||
        (t.grad_dtype != MOE_F32 && t.grad_dtype != MOE_BF16))
      return MOE_EUNSUPPORTED;
    if ((uint64_t)t.n > adamw_max_elements() || (n += (uint64_t)t.n) > adamw_max_elements())
      return MOE_EUNSUPPORTED;
    if (t.n == 0) continue;
    const bool q8 = hp->state_bits == 8;
    if (!t.param || !t.grad || !t.m || !t.v || (q8 && (!t.m_scale || !t.v_scale)))
      return MOE_EINVAL;
    if (!al16(t.param) || !al16(t.grad) || !al16(t.master) || !al16(t.m) || !al16(t.v) ||
        (q8 && (!al4(t.m_scale) || !al4(t.v_scale))))
      return MOE_EALIGN;
  }
  return launch_adamw(hp, tensors, n_tensors, state, grad_scale, lr_scale, (hipStream_t)stream);
}

}  // extern "C"
