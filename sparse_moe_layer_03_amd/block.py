"""ctypes binding of the operators around the layer (include/moe_block.h):
other selection rules for its router, its experts in 8-bit integers, and the
norms before and after a block.

Each ``moe_*`` function has the name of the C entry point it calls and takes
torch tensors.  As in ``train``, the library checks sizes and alignment, the
binding what only it can see: that every tensor lies on one GPU, is laid out as
the call reads it, and is as large as the shape says.  Calls run on the
tensors' device, on its current stream unless ``stream`` names another.
"""

from __future__ import annotations

import ctypes

import torch

from . import binding as B
from . import train as T
from .train import _DTYPE, _dtype_code, _need, _on, _workspace

SCORES = {"softmax": 0, "sigmoid": 1}

# every entry point declared in include/moe_block.h
ENTRY_POINTS = ("moe_select", "moe_route_select", "moe_select_backward", "moe_layer_backward_select",
                "moe_quantize_rows", "moe_matmul_i8_workspace_bytes", "moe_matmul_i8",
                "moe_expert_ffn_i8_workspace_bytes", "moe_expert_ffn_i8", "moe_norm_residual",
                "moe_norm_residual_backward_workspace_bytes", "moe_norm_residual_backward")


class MoeSelectParams(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("score", "n_groups", "top_groups", "group_best", "renorm")] + \
               [("renorm_eps", ctypes.c_float)]


class MoeQuantShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "M", "K", "reserved")] + \
               [("ldx", ctypes.c_int64), ("ldq", ctypes.c_int64)]


class MoeI8Shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("out_dtype", "n_groups", "M", "N", "K", "reserved")] + \
               [("lda", ctypes.c_int64), ("ldc", ctypes.c_int64)]


_FFN_IO = ("x", "xq", "x_scale", "perm", "offsets", "w_gate", "w_up", "w_down", "s_gate", "s_up", "s_down",
           "y_perm")


class MoeFfnI8IO(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _FFN_IO]


class MoeNormShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "d_model", "dtype", "rows_per_gate")] + \
               [("eps", ctypes.c_float), ("res_scale", ctypes.c_float)]


class MoeRows(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("ld", ctypes.c_int64)]


class MoeNormIO(ctypes.Structure):
    _fields_ = [("x", MoeRows), ("y", MoeRows), ("w_post", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("r", MoeRows), ("h", MoeRows), ("q", ctypes.c_void_p),
                ("q_scale", ctypes.c_void_p)]


class MoeNormGradIO(ctypes.Structure):
    _fields_ = [("r", MoeRows), ("y", MoeRows), ("w_post", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p), ("dr", MoeRows), ("dh", MoeRows), ("dx", MoeRows), ("dy", MoeRows),
                ("dgate", ctypes.c_void_p), ("dw_post", ctypes.c_void_p), ("dw_pre", ctypes.c_void_p),
                ("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = T.lib()
        vp, i64, sp = ctypes.c_void_p, ctypes.c_int64, ctypes.POINTER(B.MoeShape)
        pp = ctypes.POINTER(MoeSelectParams)
        L.moe_select.argtypes = [sp, pp, vp, i64] + [vp] * 4
        L.moe_route_select.argtypes = [sp, pp] + [vp] * 9
        L.moe_select_backward.argtypes = [sp, pp, vp, i64] + [vp] * 4
        L.moe_layer_backward_select.argtypes = [sp, pp, ctypes.POINTER(T.MoeBackwardIO), vp, vp]
        L.moe_quantize_rows.argtypes = [ctypes.POINTER(MoeQuantShape)] + [vp] * 4
        L.moe_matmul_i8_workspace_bytes.argtypes = [ctypes.POINTER(MoeI8Shape)]
        L.moe_matmul_i8.argtypes = [ctypes.POINTER(MoeI8Shape)] + [vp] * 8
        L.moe_expert_ffn_i8_workspace_bytes.argtypes = [sp]
        L.moe_expert_ffn_i8.argtypes = [sp, ctypes.POINTER(MoeFfnI8IO), vp, vp]
        L.moe_norm_residual.argtypes = [ctypes.POINTER(MoeNormShape), ctypes.POINTER(MoeNormIO), vp]
        L.moe_norm_residual_backward_workspace_bytes.argtypes = [ctypes.POINTER(MoeNormShape)]
        L.moe_norm_residual_backward.argtypes = [ctypes.POINTER(MoeNormShape), ctypes.POINTER(MoeNormGradIO),
                                                 vp, vp]
        for n in ENTRY_POINTS:
            getattr(L, n).restype = ctypes.c_size_t if n.endswith("_bytes") else ctypes.c_int
        _lib = L
    return _lib


def _matrix(name, t, dtype, rows, width, device):
    """t holds rows x width values, each row contiguous; returns the elements
    between rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name}: a tensor on {device or 'a GPU'} is needed")
    if t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, needed {dtype}")
    shape, stride = t.shape, t.stride()
    ld = stride[0] if len(shape) == 2 and shape[0] > 1 else width
    if len(shape) != 2 or shape[0] < rows or shape[1] != width or (width > 1 and stride[1] != 1) or ld < width:
        raise ValueError(f"{name}: shape {tuple(shape)} strides {stride}, needed [{rows}, {width}] in whole rows")
    return ld


def _apart(outs, ins=(), same=()):
    """No output overlaps another or an input; pairs in `same` may be one and
    the same memory (equal start and strides)."""
    def span(t):
        n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride())) if t.numel() else 0
        return t.data_ptr(), t.data_ptr() + n * t.element_size()

    outs = [(n, t) for n, t in outs if t is not None]
    ins = [(n, t) for n, t in ins if t is not None]
    for i, (n, t) in enumerate(outs):
        a0, a1 = span(t)
        for m, u in outs[i + 1:] + ins:
            b0, b1 = span(u)
            if a0 < b1 and b0 < a1:
                if (n, m) in same and a0 == b0 and t.shape == u.shape and t.stride() == u.stride():
                    continue
                raise ValueError(f"{n} and {m} overlap")


# ---- selection of experts


def make_select(score="softmax", n_groups=1, top_groups=None, group_best=1, renorm=False,
                renorm_eps=0.0) -> MoeSelectParams:
    """score: "softmax" or "sigmoid"; n_groups groups of neighbouring experts of
    which a token may select from top_groups (default all), ranked by the sum of
    their group_best (1 or 2) best keys; renorm divides the gates by their sum
    + renorm_eps."""
    return MoeSelectParams(SCORES.get(score, score), n_groups, n_groups if top_groups is None else top_groups,
                           group_best, int(bool(renorm)), renorm_eps)


def _check_select(s, logits, topk_idx, other, other_name, bias=None):
    E, Tk = s.n_ffn + s.n_zero, s.T * s.top_k
    if s.T < 1 or E < 1:
        return logits.device, E     # (the library refuses it)
    ld = _matrix("logits", logits, torch.float32, s.T, E, None)
    dev = logits.device
    _need("topk_idx", topk_idx, torch.int32, Tk, dev)
    _need(other_name, other, torch.float32, Tk, dev)
    if bias is not None:
        _need("bias", bias, torch.float32, E, dev)
    return dev, ld


def moe_select(shape: B.MoeShape, params: MoeSelectParams, logits, bias, topk_idx, topk_gate, stream=None):
    """topk_idx, topk_gate of the experts that logits [T, E] and bias select."""
    dev, ld = _check_select(shape, logits, topk_idx, topk_gate, "topk_gate", bias)
    _apart([("topk_idx", topk_idx), ("topk_gate", topk_gate)], [("logits", logits), ("bias", bias)])
    B._check("moe_select", _on(dev, lambda st: lib().moe_select(
        ctypes.byref(shape), ctypes.byref(params), B._p(logits), ld, B._p(bias), B._p(topk_idx),
        B._p(topk_gate), st), stream))


def moe_route_select(shape: B.MoeShape, params: MoeSelectParams, x, w_router, logit_bias, bias, topk_idx,
                     topk_gate, logits_out, ws, stream=None):
    """binding.moe_route with another selection rule; logits_out is needed."""
    s, E = shape, shape.n_ffn + shape.n_zero
    dev = x.device
    if s.dtype in _DTYPE and s.T >= 1:
        _need("x", x, _DTYPE[s.dtype], s.T * s.d_model)
        _need("w_router", w_router, _DTYPE[s.dtype], E * s.d_model, dev)
        _check_select(s, logits_out, topk_idx, topk_gate, "topk_gate", bias)
        _need("logits_out", logits_out, torch.float32, s.T * E, dev)
        if logit_bias is not None:
            _need("logit_bias", logit_bias, torch.float32, E, dev)

    def call(st):
        _workspace(ws, B.moe_workspace_bytes(s), dev)
        return lib().moe_route_select(ctypes.byref(s), ctypes.byref(params), B._p(x), B._p(w_router),
                                      B._p(logit_bias), B._p(bias), B._p(topk_idx), B._p(topk_gate),
                                      B._p(logits_out), B._p(ws), st)

    B._check("moe_route_select", _on(dev, call, stream))


def moe_select_backward(shape: B.MoeShape, params: MoeSelectParams, logits, topk_idx, dgate, dlogits, stream=None):
    """dlogits [T, E] from the gradient dgate [T, top_k] at topk_gate."""
    dev, ld = _check_select(shape, logits, topk_idx, dgate, "dgate")
    _need("dlogits", dlogits, torch.float32, shape.T * (shape.n_ffn + shape.n_zero), dev)
    _apart([("dlogits", dlogits)], [("logits", logits), ("topk_idx", topk_idx), ("dgate", dgate)])
    B._check("moe_select_backward", _on(dev, lambda st: lib().moe_select_backward(
        ctypes.byref(shape), ctypes.byref(params), B._p(logits), ld, B._p(topk_idx), B._p(dgate),
        B._p(dlogits), st), stream))


def moe_layer_backward_select(shape: B.MoeShape, params: MoeSelectParams, io: T.BackwardIO, ws, stream=None):
    """train.moe_layer_backward of a layer whose experts moe_select chose."""
    io.check(shape)
    dev = io.tensors["x"].device

    def call(st):
        _workspace(ws, T.moe_layer_backward_workspace_bytes(shape), dev)
        return lib().moe_layer_backward_select(ctypes.byref(shape), ctypes.byref(params), ctypes.byref(io.c),
                                               B._p(ws), st)

    B._check("moe_layer_backward_select", _on(dev, call, stream))


# ---- products in 8-bit integers


def make_quant_shape(dtype, M, K, ldx=None, ldq=None) -> MoeQuantShape:
    return MoeQuantShape(_dtype_code(dtype), M, K, 0, K if ldx is None else ldx, K if ldq is None else ldq)


def moe_quantize_rows(shape: MoeQuantShape, x, q, scale, stream=None):
    """q [M, K] int8 and scale [M]: x's rows in 8-bit codes."""
    s = shape
    if s.dtype in _DTYPE and s.M >= 0:
        T._rows("x", x, _DTYPE[s.dtype], s.M, s.K, s.ldx, x.device)
        T._rows("q", q, torch.int8, s.M, s.K, s.ldq, x.device)
        _need("scale", scale, torch.float32, s.M, x.device)
        _apart([("q", q), ("scale", scale)], [("x", x)])
    B._check("moe_quantize_rows", _on(x.device, lambda st: lib().moe_quantize_rows(
        ctypes.byref(s), B._p(x), B._p(q), B._p(scale), st), stream))


def quantize_rows(x, stream=None):
    """Codes and scales of x [..., K], contiguous, in new tensors: weights
    [n, out, in] get a scale for each output channel."""
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    scale = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
    K = x.shape[-1]
    moe_quantize_rows(make_quant_shape(x.dtype, x.numel() // K, K), x.view(-1, K), q.view(-1, K),
                      scale.view(-1), stream)
    return q, scale


def make_i8_shape(out_dtype, n_groups, M, N, K, lda=None, ldc=None) -> MoeI8Shape:
    """lda, ldc: elements between rows of a [M, K] and c [M, N] (default:
    contiguous)."""
    return MoeI8Shape(_dtype_code(out_dtype), n_groups, M, N, K, 0, K if lda is None else lda,
                      N if ldc is None else ldc)


def moe_matmul_i8_workspace_bytes(shape: MoeI8Shape) -> int:
    return int(lib().moe_matmul_i8_workspace_bytes(ctypes.byref(shape)))


def moe_matmul_i8(shape: MoeI8Shape, offsets, a, a_scale, w, w_scale, out, ws=None, stream=None):
    """out[p] = (a[p] w_e^T) a_scale[p] w_scale[e] for the rows p of group e;
    offsets None: one group of all rows."""
    s = shape
    dev = w.device
    if s.out_dtype in _DTYPE and s.M >= 0 and s.n_groups >= 1:
        if offsets is not None:
            _need("offsets", offsets, torch.int32, s.n_groups + 1, dev)
        T._rows("a", a, torch.int8, s.M, s.K, s.lda, dev)
        _need("a_scale", a_scale, torch.float32, s.M, dev)
        _need("w", w, torch.int8, s.n_groups * s.N * s.K, dev)
        _need("w_scale", w_scale, torch.float32, s.n_groups * s.N, dev)
        T._rows("out", out, _DTYPE[s.out_dtype], s.M, s.N, s.ldc, dev)
        _apart([("out", out)], [("a", a), ("a_scale", a_scale), ("w", w), ("w_scale", w_scale), ("offsets", offsets)])

    def call(st):
        _workspace(ws, moe_matmul_i8_workspace_bytes(s), dev)
        return lib().moe_matmul_i8(ctypes.byref(s), B._p(offsets), B._p(a), B._p(a_scale), B._p(w), B._p(w_scale),
                                   B._p(out), B._p(ws), st)

    B._check("moe_matmul_i8", _on(dev, call, stream))


class FfnI8IO:
    """The arrays of one pass of the experts' FFN in 8-bit integers; keeps its
    tensors alive.  The tokens come as x, or as their codes xq and x_scale."""

    def __init__(self, *, perm, offsets, w_gate, s_gate, w_up, s_up, w_down, s_down, y_perm, x=None, xq=None,
                 x_scale=None):
        given = locals()
        self.tensors = {n: given[n] for n in _FFN_IO}
        self.c = MoeFfnI8IO(*[B._p(self.tensors[n]) for n in _FFN_IO])

    def check(self, s: B.MoeShape):
        t, dt, f32, i32, i8 = self.tensors, _DTYPE.get(s.dtype), torch.float32, torch.int32, torch.int8
        if dt is None:
            return
        Tk, w, dev = s.T * s.top_k, s.n_ffn * s.d_ff * s.d_model, self.device
        need = dict(x=(dt, s.T * s.d_model), xq=(i8, s.T * s.d_model), x_scale=(f32, s.T), perm=(i32, Tk),
                    offsets=(i32, s.n_ffn + s.n_zero + 1), w_gate=(i8, w), w_up=(i8, w), w_down=(i8, w),
                    s_gate=(f32, s.n_ffn * s.d_ff), s_up=(f32, s.n_ffn * s.d_ff),
                    s_down=(f32, s.n_ffn * s.d_model), y_perm=(dt, Tk * s.d_model))
        for n, (d, k) in need.items():
            if t[n] is None and n in ("x", "xq", "x_scale"):
                continue
            _need(n, t[n], d, k, dev)
        _apart([("y_perm", t["y_perm"])], [(n, t[n]) for n in _FFN_IO[:-1]])

    @property
    def device(self):
        return self.tensors["w_gate"].device


def moe_expert_ffn_i8_workspace_bytes(shape: B.MoeShape) -> int:
    return int(lib().moe_expert_ffn_i8_workspace_bytes(ctypes.byref(shape)))


def moe_expert_ffn_i8(shape: B.MoeShape, io: FfnI8IO, ws, stream=None):
    """binding.moe_expert_ffn with 8-bit weights and rows; fills io's y_perm."""
    io.check(shape)

    def call(st):
        _workspace(ws, moe_expert_ffn_i8_workspace_bytes(shape), io.device)
        return lib().moe_expert_ffn_i8(ctypes.byref(shape), ctypes.byref(io.c), B._p(ws), st)

    B._check("moe_expert_ffn_i8", _on(io.device, call, stream))


# ---- norms around a block


def make_norm_shape(T_, d_model, dtype, eps=1e-6, res_scale=1.0, rows_per_gate=None) -> MoeNormShape:
    """rows_per_gate: tokens that share a gate row (default: all)."""
    return MoeNormShape(T_, d_model, _dtype_code(dtype), max(T_, 1) if rows_per_gate is None else rows_per_gate,
                        eps, res_scale)


def _norm_arrays(s, matrices, vectors, gates):
    """Checks the arrays of a norm call; (moe_rows by name, device)."""
    given = [t for t in (*matrices.values(), *vectors.values(), *gates.values()) if t is not None]
    if not given:
        raise ValueError("no tensors")
    dev, dt = given[0].device, _DTYPE.get(s.dtype)
    rows = {}
    for n, t in matrices.items():
        ld = 0
        if t is not None and dt is not None:
            ld = _matrix(n, t, dt, s.T, s.d_model, dev)
        rows[n] = MoeRows(B._p(t), ld)
    n_gates = -(-s.T // s.rows_per_gate) if s.rows_per_gate > 0 else 0
    for group, count in ((vectors, 1), (gates, n_gates)):
        for n, t in group.items():
            if t is not None and dt is not None:
                _need(n, t, dt, count * s.d_model, dev)
    return rows, dev


def moe_norm_residual(shape: MoeNormShape, *, x=None, y=None, w_post=None, gate=None, w_pre=None, r=None, h=None,
                      q=None, q_scale=None, stream=None):
    """r = res_scale x + gate norm(y, w_post), h = norm(r, w_pre), and h's 8-bit
    codes q with q_scale; what is None falls out (see the header)."""
    s = shape
    rows, dev = _norm_arrays(s, dict(x=x, y=y, r=r, h=h), dict(w_post=w_post, w_pre=w_pre), dict(gate=gate))
    if q is not None:
        _need("q", q, torch.int8, s.T * s.d_model, dev)
    if q_scale is not None:
        _need("q_scale", q_scale, torch.float32, s.T, dev)
    _apart([("r", r), ("h", h), ("q", q), ("q_scale", q_scale)],
           [("x", x), ("y", y), ("w_post", w_post), ("gate", gate), ("w_pre", w_pre)], {("r", "x")})
    io = MoeNormIO(rows["x"], rows["y"], B._p(w_post), B._p(gate), B._p(w_pre), rows["r"], rows["h"], B._p(q),
                   B._p(q_scale))
    B._check("moe_norm_residual", _on(dev, lambda st: lib().moe_norm_residual(
        ctypes.byref(s), ctypes.byref(io), st), stream))


def moe_norm_residual_backward_workspace_bytes(shape: MoeNormShape) -> int:
    return int(lib().moe_norm_residual_backward_workspace_bytes(ctypes.byref(shape)))


def moe_norm_residual_backward(shape: MoeNormShape, ws, *, r=None, y=None, w_post=None, gate=None, w_pre=None,
                               dr=None, dh=None, dx=None, dy=None, dgate=None, dw_post=None, dw_pre=None,
                               accumulate=False, stream=None):
    """Gradients of moe_norm_residual from dr and dh, the gradients at r and h;
    r, y and the vectors as the forward pass left and had them."""
    s = shape
    rows, dev = _norm_arrays(s, dict(r=r, y=y, dr=dr, dh=dh, dx=dx, dy=dy),
                             dict(w_post=w_post, w_pre=w_pre, dw_post=dw_post, dw_pre=dw_pre),
                             dict(gate=gate, dgate=dgate))
    _apart([("dx", dx), ("dy", dy), ("dgate", dgate), ("dw_post", dw_post), ("dw_pre", dw_pre)],
           [("r", r), ("y", y), ("w_post", w_post), ("gate", gate), ("w_pre", w_pre), ("dr", dr), ("dh", dh)],
           {(o, i) for o in ("dx", "dy") for i in ("r", "y", "dr", "dh")})
    io = MoeNormGradIO(rows["r"], rows["y"], B._p(w_post), B._p(gate), B._p(w_pre), rows["dr"], rows["dh"],
                       rows["dx"], rows["dy"], B._p(dgate), B._p(dw_post), B._p(dw_pre), int(bool(accumulate)), 0)

    def call(st):
        _workspace(ws, moe_norm_residual_backward_workspace_bytes(s), dev)
        return lib().moe_norm_residual_backward(ctypes.byref(s), ctypes.byref(io), B._p(ws), st)

    B._check("moe_norm_residual_backward", _on(dev, call, stream))
