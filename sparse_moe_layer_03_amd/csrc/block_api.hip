// C ABI of the operators around the layer (moe_block.h): argument checks,
// workspace layout and the launch sequence of each call.  Every check runs on
// the host before any work is enqueued; no call allocates, frees or
// synchronises.

#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "block.h"
#include "common.h"

namespace moe {

static bool al16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static bool al4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
static size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }
static int elem_size(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }

static int check_select(const moe_shape* s, const moe_select_params* p) {
  const int rc = check_shape(s);
  if (rc) return rc;
  if (p == nullptr) return MOE_EINVAL;
  const int E = s->n_ffn + s->n_zero;
  if (p->score != MOE_SCORE_SOFTMAX && p->score != MOE_SCORE_SIGMOID) return MOE_EINVAL;
  if (p->n_groups < 1 || E % p->n_groups != 0 || p->top_groups < 1 || p->top_groups > p->n_groups ||
      (p->group_best != 1 && p->group_best != 2) || p->group_best > E / p->n_groups ||
      s->top_k > p->top_groups * (E / p->n_groups))
    return MOE_EINVAL;
  if (!isfinite(p->renorm_eps)) return MOE_ENONFINITE;
  if (p->renorm_eps < 0.f) return MOE_EINVAL;
  if (p->n_groups > 64 || (long)s->T * s->top_k >= kGmmMaxRows) return MOE_EUNSUPPORTED;
  return MOE_OK;
}

static int run_select(const moe_shape* s, const moe_select_params* p, const float* logits,
                      int64_t ld, const float* bias, int32_t* idx, float* gate, hipStream_t st) {
  SelectArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.bias = bias;
  a.idx = idx;
  a.gate = gate;
  a.scaling = s->routed_scaling;
  a.eps = p->renorm_eps;
  a.T = s->T;
  a.E = s->n_ffn + s->n_zero;
  a.k = s->top_k;
  a.score = p->score;
  a.n_groups = p->n_groups;
  // (all groups stay: one group)
  if (p->top_groups == p->n_groups) a.n_groups = 1;
  a.top_groups = a.n_groups == 1 ? 1 : p->top_groups;
  a.group_best = p->group_best;
  a.renorm = p->renorm != 0;
  return launch_select(a, st);
}

static int check_quant(const moe_quant_shape* s) {
  if (s == nullptr) return MOE_EINVAL;
  if (s->M < 0 || s->K < 1 || s->ldx < s->K || s->ldq < s->K || s->reserved != 0) return MOE_EINVAL;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) return MOE_EUNSUPPORTED;
  if (s->M >= kGmmMaxRows || s->K >= (1 << 17) || s->ldx >= (1 << 24) || s->ldq >= (1 << 24))
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

static int check_i8(const moe_i8_shape* s) {
  if (s == nullptr) return MOE_EINVAL;
  if (s->n_groups < 1 || s->M < 0 || s->N < 1 || s->K < 1 || s->lda < s->K || s->ldc < s->N ||
      s->reserved != 0)
    return MOE_EINVAL;
  if (s->out_dtype != MOE_F32 && s->out_dtype != MOE_BF16) return MOE_EUNSUPPORTED;
  if (s->n_groups > 1024 || s->M >= kGmmMaxRows || s->N > (1 << 20) || s->K >= (1 << 17) ||
      s->lda >= (1 << 24) || s->ldc >= (1 << 24))
    return MOE_EUNSUPPORTED;
  return MOE_OK;
}

// A product with too few tiles to give every second CU one has its reduction cut
// into as many ranges, of at least 512 codes each, as make three tiles for two
// CUs; their sums are joined by a second kernel.  us without, and with 4, 8 and 16
// ranges: 128 x 2048 of K 8192 39, 20.9, 19.2, 22.5; 256 x 1024 of 16384 68, 29,
// 22.5, 25; 16 x 2048 of 8192 41, 17, 13.5, 12.6; 128 x 4096 of 4096 23, 19, 22,
// 22; and with more tiles 512 x 2048 of 4096 24, 24, 30, 29.  A function of the
// sizes and the device's CU count only: it sizes the workspace.
static int i8_nsplit(const moe_i8_shape* s, int cus) {
  const long G = s->n_groups, M = s->M;
  // the smallest tiles of the kernels
  const long wide = i8_mfma_ok(s->N, s->K, s->lda, s->ldc) ? 128 : 64;
  const long tiles = (M / 64 + std::min(G, M)) * ((s->N + wide - 1) / wide);
  if (tiles < 1 || 2 * tiles > cus) return 1;
  return (int)std::max(1l, std::min({32l, 3l * cus / (2 * tiles), (long)s->K / 512}));
}

static size_t i8_part_bytes(const moe_i8_shape* s, int nsplit) {
  return nsplit > 1 ? up256((size_t)nsplit * s->M * s->N * 4) : 0;
}

static int run_i8(int out_dtype, const I8Args& g, hipStream_t st) {
  const int rc = i8_mfma_ok(g.N, g.K, g.lda, g.ldo) ? launch_i8_mfma(out_dtype, g, st)
                                                    : launch_i8_general(out_dtype, g, st);
  if (rc || g.nsplit <= 1) return rc;
  return launch_i8_join(out_dtype, g, st);
}

// ---- the experts' FFN in 8-bit integers: workspace

struct FfnLayout {
  size_t xq, xs, tok, rs, h, hq, hs, total;
};

static FfnLayout ffn_layout(const moe_shape* s) {
  const size_t rows = (size_t)s->T * s->top_k, d = s->d_model, f = s->d_ff;
  FfnLayout w;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = up256(off + bytes);
    return at;
  };
  w.xq = take((size_t)s->T * d);
  w.xs = take((size_t)s->T * 4);
  w.tok = take(rows * 4);
  w.rs = take(rows * 4);
  w.h = take(rows * f * elem_size(s->dtype));
  w.hq = take(rows * f);
  w.hs = take(rows * 4);
  w.total = off;
  return w;
}

static int check_ffn(const moe_shape* s) {
  const int rc = check_shape(s);
  if (rc) return rc;
  // (the tokens' codes are addressed by 31-bit offsets)
  return (long)s->T * s->top_k < kGmmMaxRows && s->d_model < (1 << 17) && s->d_ff < (1 << 17) &&
                 (long)s->T * s->d_model < (1l << 31) - (1 << 16)
             ? MOE_OK
             : MOE_EUNSUPPORTED;
}

// ---- norms

static int check_norm(const moe_norm_shape* s) {
  if (s == nullptr) return MOE_EINVAL;
  if (s->T < 0 || s->d_model < 1 || s->rows_per_gate < 1) return MOE_EINVAL;
  if (s->dtype != MOE_F32 && s->dtype != MOE_BF16) return MOE_EUNSUPPORTED;
  if (s->T >= kGmmMaxRows || s->d_model > 32768) return MOE_EUNSUPPORTED;
  if (!isfinite(s->eps) || !isfinite(s->res_scale)) return MOE_ENONFINITE;
  if (s->eps < 0.f) return MOE_EINVAL;
  return MOE_OK;
}

static int check_rows(const moe_norm_shape* s, const moe_rows& r) {
  if (r.p == nullptr) return MOE_OK;
  if (r.ld < s->d_model) return MOE_EINVAL;
  if (r.ld >= (1 << 24)) return MOE_EUNSUPPORTED;
  return al16(r.p) ? MOE_OK : MOE_EALIGN;
}

}  // namespace moe

using namespace moe;

extern "C" {

int moe_select(const moe_shape* s, const moe_select_params* p, const float* logits,
               int64_t ld_logits, const float* bias, int32_t* topk_idx, float* topk_gate,
               void* stream) {
  const int rc = check_select(s, p);
  if (rc) return rc;
  if (!logits || !topk_idx || !topk_gate || ld_logits < s->n_ffn + s->n_zero) return MOE_EINVAL;
  if (ld_logits >= (1 << 24)) return MOE_EUNSUPPORTED;
  if (!al4(logits) || !al4(bias) || !al4(topk_idx) || !al4(topk_gate)) return MOE_EALIGN;
  const size_t T = s->T, E = (size_t)s->n_ffn + s->n_zero;
  Arrays v;
  v.rows(logits, ld_logits, s->T, (int)E, 4, false, false);
  v.add(bias, E * 4, false);
  v.add(topk_idx, T * s->top_k * 4, true);
  v.add(topk_gate, T * s->top_k * 4, true);
  if (const int bad = v.check()) return bad;
  return run_select(s, p, logits, ld_logits, bias, topk_idx, topk_gate, (hipStream_t)stream);
}

int moe_route_select(const moe_shape* s, const moe_select_params* p, const void* x,
                     const void* w_router, const float* logit_bias, const float* bias,
                     int32_t* topk_idx, float* topk_gate, float* logits_out, void* ws,
                     void* stream) {
  int rc = check_select(s, p);
  if (rc) return rc;
  if (!x || !w_router || !topk_idx || !topk_gate || !logits_out || !ws) return MOE_EINVAL;
  if (!al16(x) || !al16(w_router) || !al16(ws) || !al4(logit_bias) || !al4(bias) ||
      !al4(topk_idx) || !al4(topk_gate) || !al4(logits_out))
    return MOE_EALIGN;
  const size_t T = s->T, E = (size_t)s->n_ffn + s->n_zero, d = s->d_model, es = elem_size(s->dtype);
  Arrays v;
  v.add(x, T * d * es, false);
  v.add(w_router, E * d * es, false);
  v.add(logit_bias, E * 4, false);
  v.add(bias, E * 4, false);
  v.add(topk_idx, T * s->top_k * 4, true);
  v.add(topk_gate, T * s->top_k * 4, true);
  v.add(logits_out, T * E * 4, true);
  v.add(ws, moe_workspace_bytes(s), true);
  if ((rc = v.check())) return rc;
  if ((rc = run_router_logits(s, x, w_router, logit_bias, logits_out, ws, (hipStream_t)stream)))
    return rc;
  return run_select(s, p, logits_out, s->n_ffn + s->n_zero, bias, topk_idx, topk_gate,
                    (hipStream_t)stream);
}

int moe_select_backward(const moe_shape* s, const moe_select_params* p, const float* logits,
                        int64_t ld_logits, const int32_t* topk_idx, const float* dgate,
                        float* dlogits, void* stream) {
  const int rc = check_select(s, p);
  if (rc) return rc;
  if (!logits || !topk_idx || !dgate || !dlogits || ld_logits < s->n_ffn + s->n_zero)
    return MOE_EINVAL;
  if (ld_logits >= (1 << 24)) return MOE_EUNSUPPORTED;
  if (!al4(logits) || !al4(topk_idx) || !al4(dgate) || !al4(dlogits)) return MOE_EALIGN;
  const size_t T = s->T, E = (size_t)s->n_ffn + s->n_zero;
  Arrays v;
  v.rows(logits, ld_logits, s->T, (int)E, 4, false, false);
  v.add(topk_idx, T * s->top_k * 4, false);
  v.add(dgate, T * s->top_k * 4, false);
  v.add(dlogits, T * E * 4, true);
  if (const int bad = v.check()) return bad;
  SelectBwdArgs a{};
  a.logits = logits;
  a.ld = ld_logits;
  a.idx = topk_idx;
  a.dgate = dgate;
  a.dlogits = dlogits;
  a.scaling = s->routed_scaling;
  a.eps = p->renorm_eps;
  a.T = s->T;
  a.E = s->n_ffn + s->n_zero;
  a.k = s->top_k;
  a.score = p->score;
  a.renorm = p->renorm != 0;
  return launch_select_bwd(a, (hipStream_t)stream);
}

int moe_layer_backward_select(const moe_shape* s, const moe_select_params* p,
                              const moe_backward_io* io, void* ws, void* stream) {
  const int rc = check_select(s, p);
  if (rc) return rc;
  if (!io || !io->logits) return MOE_EINVAL;
  return run_layer_backward(s, p, io, ws, (hipStream_t)stream);
}

int moe_quantize_rows(const moe_quant_shape* s, const void* x, int8_t* q, float* scale,
                      void* stream) {
  const int rc = check_quant(s);
  if (rc) return rc;
  if (s->M > 0 && (!x || !q || !scale)) return MOE_EINVAL;
  if (!al16(x) || !al16(q) || !al4(scale)) return MOE_EALIGN;
  Arrays v;
  v.rows(x, s->ldx, s->M, s->K, elem_size(s->dtype), false, false);
  v.rows(q, s->ldq, s->M, s->K, 1, true, false);
  v.add(scale, (size_t)s->M * 4, true);
  if (const int bad = v.check()) return bad;
  return launch_quantize(s->dtype, x, s->ldx, s->M, s->K, q, s->ldq, scale, nullptr,
                         (hipStream_t)stream);
}

size_t moe_matmul_i8_workspace_bytes(const moe_i8_shape* s) {
  if (check_i8(s) != MOE_OK) return 0;
  const int cus = device_cu_count();
  return cus > 0 ? i8_part_bytes(s, i8_nsplit(s, cus)) : 0;
}

int moe_matmul_i8(const moe_i8_shape* s, const int32_t* offsets, const int8_t* a,
                  const float* a_scale, const int8_t* w, const float* w_scale, void* c, void* ws,
                  void* stream) {
  const int rc = check_i8(s);
  if (rc) return rc;
  const bool none = s->M == 0;
  if ((!offsets && s->n_groups > 1) || !w || !w_scale || (!none && (!a || !a_scale || !c)))
    return MOE_EINVAL;
  if (!al4(offsets) || !al16(a) || !al4(a_scale) || !al16(w) || !al4(w_scale) || !al16(c) || !al16(ws))
    return MOE_EALIGN;
  const int cus = device_cu_count();
  if (cus <= 0) return MOE_EHIP;
  I8Args g{};
  g.nsplit = i8_nsplit(s, cus);
  if (g.nsplit > 1 && !ws) return MOE_EINVAL;
  if (none) return MOE_OK;
  Arrays v;
  v.rows(a, s->lda, s->M, s->K, 1, false, false);
  v.add(a_scale, (size_t)s->M * 4, false);
  v.add(w, (size_t)s->n_groups * s->N * s->K, false);
  v.add(w_scale, (size_t)s->n_groups * s->N * 4, false);
  v.add(offsets, ((size_t)s->n_groups + 1) * 4, false);
  v.rows(c, s->ldc, s->M, s->N, elem_size(s->out_dtype), true, false);
  v.add(ws, i8_part_bytes(s, g.nsplit), true);
  if (const int bad = v.check()) return bad;
  g.a = a;
  g.sa = a_scale;
  g.b = w;
  g.sb = w_scale;
  g.out = c;
  g.offsets = offsets;
  g.lda = s->lda;
  g.ldo = s->ldc;
  g.ngroups = s->n_groups;
  g.M = g.rows = s->M;
  g.N = s->N;
  g.K = s->K;
  g.part = (int32_t*)ws;
  return run_i8(s->out_dtype, g, (hipStream_t)stream);
}

size_t moe_expert_ffn_i8_workspace_bytes(const moe_shape* s) {
  return check_ffn(s) == MOE_OK ? ffn_layout(s).total : 0;
}

int moe_expert_ffn_i8(const moe_shape* s, const moe_ffn_i8_io* io, void* ws, void* stream) {
  int rc = check_ffn(s);
  if (rc) return rc;
  if (!io || !ws) return MOE_EINVAL;
  if ((io->xq ? !io->x_scale || io->x : !io->x || io->x_scale) || !io->perm || !io->offsets ||
      !io->w_gate || !io->w_up || !io->w_down || !io->s_gate || !io->s_up || !io->s_down || !io->y_perm)
    return MOE_EINVAL;
  if (!al16(io->x) || !al16(io->xq) || !al4(io->x_scale) || !al4(io->perm) || !al4(io->offsets) ||
      !al16(io->w_gate) || !al16(io->w_up) || !al16(io->w_down) || !al4(io->s_gate) ||
      !al4(io->s_up) || !al4(io->s_down) || !al16(io->y_perm) || !al16(ws))
    return MOE_EALIGN;
  hipStream_t st = (hipStream_t)stream;
  const FfnLayout w = ffn_layout(s);
  {
    const size_t T = s->T, rows = T * s->top_k, dd = s->d_model, es = elem_size(s->dtype);
    const size_t up = (size_t)s->n_ffn * s->d_ff * dd, E = (size_t)s->n_ffn + s->n_zero;
    Arrays v;
    v.add(io->x, T * dd * es, false);
    v.add(io->xq, T * dd, false);
    v.add(io->x_scale, T * 4, false);
    v.add(io->perm, rows * 4, false);
    v.add(io->offsets, (E + 1) * 4, false);
    v.add(io->w_gate, up, false);
    v.add(io->w_up, up, false);
    v.add(io->w_down, up, false);
    v.add(io->s_gate, (size_t)s->n_ffn * s->d_ff * 4, false);
    v.add(io->s_up, (size_t)s->n_ffn * s->d_ff * 4, false);
    v.add(io->s_down, (size_t)s->n_ffn * dd * 4, false);
    v.add(io->y_perm, rows * dd * es, true);
    v.add(ws, w.total, true);
    if ((rc = v.check())) return rc;
  }
  char* base = (char*)ws;
  const int Tk = s->T * s->top_k, d = s->d_model, f = s->d_ff;
  const int8_t* xq = io->xq;
  const float* xs = io->x_scale;
  if (!xq) {
    int8_t* q = (int8_t*)(base + w.xq);
    float* qs = (float*)(base + w.xs);
    if ((rc = launch_quantize(s->dtype, io->x, d, s->T, d, q, d, qs, nullptr, st))) return rc;
    xq = q;
    xs = qs;
  }
  int8_t* hq = (int8_t*)(base + w.hq);
  int32_t* tok = (int32_t*)(base + w.tok);
  float *rs = (float*)(base + w.rs), *hs = (float*)(base + w.hs);
  if ((rc = launch_row_tokens(xs, io->perm, io->offsets, s->n_ffn, Tk, s->top_k, tok, rs, st))) return rc;
  I8Args g{};
  g.a = xq;
  g.a_bytes = (uint32_t)((size_t)s->T * d);
  g.tok = tok;
  g.sa = rs;
  g.b = io->w_gate;
  g.b2 = io->w_up;
  g.sb = io->s_gate;
  g.sb2 = io->s_up;
  g.out = base + w.h;
  g.offsets = io->offsets;
  g.lda = d;
  g.ldo = f;
  g.ngroups = s->n_ffn;
  g.M = Tk;
  // (as many fall on FFN experts where all are chosen alike)
  g.rows = std::max(1, (int)((long)Tk * s->n_ffn / (s->n_ffn + s->n_zero)));
  g.N = f;
  g.K = d;
  g.nsplit = 1;
  if ((rc = launch_i8_mfma(s->dtype, g, st))) return rc;
  if ((rc = launch_quantize(s->dtype, base + w.h, f, Tk, f, hq, f, hs, io->offsets + s->n_ffn, st)))
    return rc;
  g.a = hq;
  g.sa = hs;
  g.b = io->w_down;
  g.b2 = nullptr;
  g.sb = io->s_down;
  g.out = io->y_perm;
  g.lda = f;
  g.ldo = d;
  g.N = d;
  g.K = f;
  return launch_i8_mfma(s->dtype, g, st);
}

int moe_norm_residual(const moe_norm_shape* s, const moe_norm_io* io, void* stream) {
  int rc = check_norm(s);
  if (rc) return rc;
  if (!io) return MOE_EINVAL;
  const bool y = io->y.p, x = io->x.p, pre = io->w_pre, none = s->T == 0;
  if (!none) {
    if (!y && (!x || io->r.p || io->w_post || io->gate || s->res_scale != 1.f || !pre)) return MOE_EINVAL;
    if (y && !io->r.p) return MOE_EINVAL;
    if (pre ? !io->h.p && !io->q : io->h.p || io->q) return MOE_EINVAL;
    if ((io->q != nullptr) != (io->q_scale != nullptr)) return MOE_EINVAL;
  }
  if ((rc = check_rows(s, io->x)) || (rc = check_rows(s, io->y)) || (rc = check_rows(s, io->r)) ||
      (rc = check_rows(s, io->h)))
    return rc;
  if (!al16(io->w_post) || !al16(io->gate) || !al16(io->w_pre) || !al16(io->q) || !al4(io->q_scale))
    return MOE_EALIGN;
  const int T = s->T, d = s->d_model, es = elem_size(s->dtype);
  const size_t vec = (size_t)d * es, gates = ((size_t)T + s->rows_per_gate - 1) / s->rows_per_gate;
  Arrays v;
  v.rows(io->x.p, io->x.ld, T, d, es, false, true);
  v.rows(io->r.p, io->r.ld, T, d, es, true, true);
  v.rows(io->y.p, io->y.ld, T, d, es, false, false);
  v.rows(io->h.p, io->h.ld, T, d, es, true, false);
  v.add(io->w_post, vec, false);
  v.add(io->gate, gates * vec, false);
  v.add(io->w_pre, vec, false);
  v.add(io->q, (size_t)T * d, true);
  v.add(io->q_scale, (size_t)T * 4, true);
  if ((rc = v.check())) return rc;
  return launch_norm(*s, *io, (hipStream_t)stream);
}

size_t moe_norm_residual_backward_workspace_bytes(const moe_norm_shape* s) {
  if (check_norm(s) != MOE_OK) return 0;
  const int cus = device_cu_count();
  return cus > 0 ? norm_bwd_ws_bytes(*s, cus) : 0;
}

int moe_norm_residual_backward(const moe_norm_shape* s, const moe_norm_grad_io* io, void* ws,
                               void* stream) {
  int rc = check_norm(s);
  if (rc) return rc;
  if (!io || !ws || io->reserved != 0) return MOE_EINVAL;
  const bool y = io->y.p, pre = io->w_pre, none = s->T == 0;
  if (!none) {
    if (pre != (io->dh.p != nullptr) || (pre && !io->r.p) || y != (io->dy.p != nullptr)) return MOE_EINVAL;
    if (!y && (io->w_post || io->gate)) return MOE_EINVAL;
    if (!io->dr.p && !pre) return MOE_EINVAL;
    if (!y && !io->dx.p && !io->dw_pre) return MOE_EINVAL;
  }
  if ((io->dgate && !io->gate) || (io->dw_post && !io->w_post) || (io->dw_pre && !io->w_pre))
    return MOE_EINVAL;
  if ((rc = check_rows(s, io->r)) || (rc = check_rows(s, io->y)) || (rc = check_rows(s, io->dr)) ||
      (rc = check_rows(s, io->dh)) || (rc = check_rows(s, io->dx)) || (rc = check_rows(s, io->dy)))
    return rc;
  if (!al16(io->w_post) || !al16(io->gate) || !al16(io->w_pre) || !al16(io->dgate) ||
      !al16(io->dw_post) || !al16(io->dw_pre) || !al16(ws))
    return MOE_EALIGN;
  const int cus = device_cu_count();
  if (cus <= 0) return MOE_EHIP;
  const int T = s->T, d = s->d_model, es = elem_size(s->dtype);
  const size_t vec = (size_t)d * es, gates = ((size_t)T + s->rows_per_gate - 1) / s->rows_per_gate;
  Arrays v;
  v.rows(io->r.p, io->r.ld, T, d, es, false, true);
  v.rows(io->y.p, io->y.ld, T, d, es, false, true);
  v.rows(io->dr.p, io->dr.ld, T, d, es, false, true);
  v.rows(io->dh.p, io->dh.ld, T, d, es, false, true);
  v.rows(io->dx.p, io->dx.ld, T, d, es, true, true);
  v.rows(io->dy.p, io->dy.ld, T, d, es, true, true);
  v.add(io->w_post, vec, false);
  v.add(io->gate, gates * vec, false);
  v.add(io->w_pre, vec, false);
  v.add(io->dgate, gates * vec, true);
  v.add(io->dw_post, vec, true);
  v.add(io->dw_pre, vec, true);
  v.add(ws, norm_bwd_ws_bytes(*s, cus), true);
  if ((rc = v.check())) return rc;
  return launch_norm_bwd(*s, *io, ws, cus, (hipStream_t)stream);
}

}  // extern "C"
