"""ctypes binding of the operators around the layer (include/moe_block.h):
other selection rules for its router, its experts in 8-bit integers, and the
norms before and after a block.

Each ``moe_*`` function has the name of the C entry point it calls and takes
torch tensors.  As in ``train``, the library checks sizes, alignment and
overlaps, the binding what only it can see: that every tensor lies on one GPU,
is laid out as the call reads it, and is as large as the shape says.  Calls run
on the tensors' device, on its current stream unless ``stream`` names another.
``block_forward`` and ``block_backward`` put the operators together with the
layer's own calls, as the blocks of a model use them.
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from . import binding as B
from . import train as T
from .train import _DTYPE, _dtype_code

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


def _rows_fields(*names):
    """moe_rows members, each as a pointer and the elements between rows."""
    return [f for n in names for f in ((n, ctypes.c_void_p), (n + "_ld", ctypes.c_int64))]


class MoeNormIO(ctypes.Structure):
    _fields_ = _rows_fields("x", "y") + [(n, ctypes.c_void_p) for n in ("w_post", "gate", "w_pre")] + \
        _rows_fields("r", "h") + [("q", ctypes.c_void_p), ("q_scale", ctypes.c_void_p)]


class MoeNormGradIO(ctypes.Structure):
    _fields_ = _rows_fields("r", "y") + [(n, ctypes.c_void_p) for n in ("w_post", "gate", "w_pre")] + \
        _rows_fields("dr", "dh", "dx", "dy") + [(n, ctypes.c_void_p) for n in ("dgate", "dw_post", "dw_pre")] + \
        [("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32)]


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


# Checks of a tensor; each returns what the call takes of it.  Small calls are
# as long as these, so they ask for as little as they can.


def _device(name, t):
    """The index of the tensor's GPU."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: a tensor on a GPU is needed")
    return t.get_device()


def _flat(name, t, dtype, numel, dev):
    """The address of a contiguous tensor of dtype on GPU dev with at least
    numel elements."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != dev or \
            t.numel() < numel or not t.is_contiguous():
        _refuse(name, t, f"{numel} contiguous elements of {dtype}", dev)
    return t.data_ptr()


def _opt(name, t, dtype, numel, dev):
    return None if t is None else _flat(name, t, dtype, numel, dev)


def _matrix(name, t, dtype, rows, width, dev):
    """Address and elements between rows of a tensor of rows x width values, each
    row contiguous; (None, 0) for None."""
    if t is None:
        return None, 0
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == dev and t.dim() == 2:
        shape, (ld, one) = t.shape, t.stride()
        if shape[0] <= 1:
            ld = width
        if shape[0] >= rows and shape[1] == width and (one == 1 or width == 1) and ld >= width:
            return t.data_ptr(), ld
    _refuse(name, t, f"[{rows}, {width}] of {dtype} in whole rows", dev)


def _refuse(name, t, need, dev):
    have = "no tensor"
    if isinstance(t, torch.Tensor):
        have = f"{tuple(t.shape)} of {t.dtype} on {t.device}, strides {t.stride()}"
    raise ValueError(f"{name}: {have}, needed {need} on cuda:{dev}")


def _scratch(ws, need, dev):
    """The address of at least `need` bytes on GPU dev (None: 0)."""
    if need and (ws is None or ws.get_device() != dev or not ws.is_contiguous()
                 or ws.numel() * ws.element_size() < need):
        raise ValueError(f"ws: {need} bytes on cuda:{dev} are needed")
    return None if ws is None else ws.data_ptr()


def _on(dev, call, *args):
    """call(*args) with GPU dev as the current one (workspaces go by its CUs)."""
    if dev == torch.cuda.current_device():
        return call(*args)
    with torch.cuda.device(dev):
        return call(*args)


def _run(name, dev, stream, *args):
    """The entry point's call on GPU dev, on `stream` or its current one."""
    fn = getattr(lib(), name)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _run(name, dev, stream, *args)
    if stream is None:
        handle = torch.cuda.current_stream(dev).cuda_stream
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device.index != dev:
            raise ValueError(f"stream: on {stream.device}, needed on cuda:{dev}")
        handle = stream.cuda_stream
    else:
        handle = int(stream)
    rc = fn(*args, handle)
    if rc:
        B._check(name, rc)


# ---- selection of experts


def make_select(score="softmax", n_groups=1, top_groups=None, group_best=1, renorm=False,
                renorm_eps=0.0) -> MoeSelectParams:
    """score: "softmax" or "sigmoid"; n_groups groups of neighbouring experts of
    which a token may select from top_groups (default all), ranked by the sum of
    their group_best (1 or 2) best keys; renorm divides the gates by their sum
    + renorm_eps."""
    return MoeSelectParams(SCORES.get(score, score), n_groups, n_groups if top_groups is None else top_groups,
                           group_best, int(bool(renorm)), renorm_eps)


def _sizes(s):
    return s.T, s.n_ffn + s.n_zero, s.T * s.top_k


def moe_select(shape: B.MoeShape, params: MoeSelectParams, logits, bias, topk_idx, topk_gate, stream=None):
    """topk_idx, topk_gate of the experts that logits [T, E] and bias select."""
    T_, E, Tk = _sizes(shape)
    dev = _device("logits", logits)
    f32 = torch.float32
    x, ld = _matrix("logits", logits, f32, T_, E, dev)
    _run("moe_select", dev, stream, ctypes.byref(shape), ctypes.byref(params), x, ld,
         _opt("bias", bias, f32, E, dev), _flat("topk_idx", topk_idx, torch.int32, Tk, dev),
         _flat("topk_gate", topk_gate, f32, Tk, dev))


def moe_route_select(shape: B.MoeShape, params: MoeSelectParams, x, w_router, logit_bias, bias, topk_idx,
                     topk_gate, logits_out, ws, stream=None):
    """binding.moe_route with another selection rule; logits_out is needed."""
    s, (T_, E, Tk) = shape, _sizes(shape)
    dev, dt, f32 = _device("x", x), _DTYPE.get(s.dtype), torch.float32
    _run("moe_route_select", dev, stream, ctypes.byref(s), ctypes.byref(params),
         _flat("x", x, dt, T_ * s.d_model, dev), _flat("w_router", w_router, dt, E * s.d_model, dev),
         _opt("logit_bias", logit_bias, f32, E, dev), _opt("bias", bias, f32, E, dev),
         _flat("topk_idx", topk_idx, torch.int32, Tk, dev), _flat("topk_gate", topk_gate, f32, Tk, dev),
         _flat("logits_out", logits_out, f32, T_ * E, dev), _scratch(ws, _on(dev, B.moe_workspace_bytes, s), dev))


def moe_select_backward(shape: B.MoeShape, params: MoeSelectParams, logits, topk_idx, dgate, dlogits, stream=None):
    """dlogits [T, E] from the gradient dgate [T, top_k] at topk_gate."""
    T_, E, Tk = _sizes(shape)
    dev = _device("logits", logits)
    f32 = torch.float32
    x, ld = _matrix("logits", logits, f32, T_, E, dev)
    _run("moe_select_backward", dev, stream, ctypes.byref(shape), ctypes.byref(params), x, ld,
         _flat("topk_idx", topk_idx, torch.int32, Tk, dev), _flat("dgate", dgate, f32, Tk, dev),
         _flat("dlogits", dlogits, f32, T_ * E, dev))


def moe_layer_backward_select(shape: B.MoeShape, params: MoeSelectParams, io: T.BackwardIO, ws, stream=None):
    """train.moe_layer_backward of a layer whose experts moe_select chose."""
    io.check(shape)
    dev = _device("x", io.tensors["x"])
    _run("moe_layer_backward_select", dev, stream, ctypes.byref(shape), ctypes.byref(params), ctypes.byref(io.c),
         _scratch(ws, _on(dev, T.moe_layer_backward_workspace_bytes, shape), dev))


# ---- products in 8-bit integers


def make_quant_shape(dtype, M, K, ldx=None, ldq=None) -> MoeQuantShape:
    return MoeQuantShape(_dtype_code(dtype), M, K, 0, K if ldx is None else ldx, K if ldq is None else ldq)


def _strided(name, t, dtype, rows, width, ld, dev):
    """The address of rows x width values, `ld` elements between rows."""
    p, have = _matrix(name, t, dtype, rows, width, dev)
    if t is not None and have != ld and t.shape[0] > 1:
        _refuse(name, t, f"{ld} elements between rows", dev)
    return p


def moe_quantize_rows(shape: MoeQuantShape, x, q, scale, stream=None):
    """q [M, K] int8 and scale [M]: x's rows in 8-bit codes."""
    s, dev = shape, _device("x", x)
    _run("moe_quantize_rows", dev, stream, ctypes.byref(s), _strided("x", x, _DTYPE.get(s.dtype), s.M, s.K, s.ldx, dev),
         _strided("q", q, torch.int8, s.M, s.K, s.ldq, dev), _flat("scale", scale, torch.float32, s.M, dev))


def _allocating_on(stream, device):
    """Tensors made inside belong to `stream` (torch's allocator hands out memory
    in the order of one stream's work); None: to the current one."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def quantize_rows(x, stream=None):
    """Codes and scales of x [..., K], contiguous, in new tensors: weights
    [n, out, in] get a scale for each output channel.  The tensors belong to
    `stream`, as if made with it as the current one: another stream that reads
    them waits for it first and marks its use (Tensor.record_stream)."""
    _device("x", x)
    with _allocating_on(stream, x.device):
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
    s, dev, f32, i8 = shape, _device("w", w), torch.float32, torch.int8
    GN = s.n_groups * s.N
    _run("moe_matmul_i8", dev, stream, ctypes.byref(s), _opt("offsets", offsets, torch.int32, s.n_groups + 1, dev),
         _strided("a", a, i8, s.M, s.K, s.lda, dev), _flat("a_scale", a_scale, f32, s.M, dev),
         _flat("w", w, i8, GN * s.K, dev), _flat("w_scale", w_scale, f32, GN, dev),
         _strided("out", out, _DTYPE.get(s.out_dtype), s.M, s.N, s.ldc, dev),
         _scratch(ws, _on(dev, moe_matmul_i8_workspace_bytes, s), dev))


class FfnI8IO:
    """The arrays of one pass of the experts' FFN in 8-bit integers; keeps its
    tensors alive.  The tokens come as x, or as their codes xq and x_scale."""

    def __init__(self, *, perm, offsets, w_gate, s_gate, w_up, s_up, w_down, s_down, y_perm, x=None, xq=None,
                 x_scale=None):
        given = locals()
        self.tensors = {n: given[n] for n in _FFN_IO}
        self.c = MoeFfnI8IO(*[B._p(self.tensors[n]) for n in _FFN_IO])

    def check(self, s: B.MoeShape, dev):
        t, f32, i8 = self.tensors, torch.float32, torch.int8
        Td, Tk, nf, w = s.T * s.d_model, s.T * s.top_k, s.n_ffn * s.d_ff, s.n_ffn * s.d_ff * s.d_model
        _opt("x", t["x"], _DTYPE.get(s.dtype), Td, dev)
        _opt("xq", t["xq"], i8, Td, dev)
        _opt("x_scale", t["x_scale"], f32, s.T, dev)
        _flat("perm", t["perm"], torch.int32, Tk, dev)
        _flat("offsets", t["offsets"], torch.int32, s.n_ffn + s.n_zero + 1, dev)
        for n, scales in (("gate", nf), ("up", nf), ("down", s.n_ffn * s.d_model)):
            _flat("w_" + n, t["w_" + n], i8, w, dev)
            _flat("s_" + n, t["s_" + n], f32, scales, dev)
        _flat("y_perm", t["y_perm"], _DTYPE.get(s.dtype), Tk * s.d_model, dev)


def moe_expert_ffn_i8_workspace_bytes(shape: B.MoeShape) -> int:
    return int(lib().moe_expert_ffn_i8_workspace_bytes(ctypes.byref(shape)))


def moe_expert_ffn_i8(shape: B.MoeShape, io: FfnI8IO, ws, stream=None):
    """binding.moe_expert_ffn with 8-bit weights and rows; fills io's y_perm."""
    dev = _device("w_gate", io.tensors["w_gate"])
    io.check(shape, dev)
    _run("moe_expert_ffn_i8", dev, stream, ctypes.byref(shape), ctypes.byref(io.c),
         _scratch(ws, moe_expert_ffn_i8_workspace_bytes(shape), dev))


# ---- norms around a block


def make_norm_shape(T_, d_model, dtype, eps=1e-6, res_scale=1.0, rows_per_gate=None) -> MoeNormShape:
    """rows_per_gate: tokens that share a gate row (default: all)."""
    return MoeNormShape(T_, d_model, _dtype_code(dtype), max(T_, 1) if rows_per_gate is None else rows_per_gate,
                        eps, res_scale)


def moe_norm_residual(shape: MoeNormShape, *, x=None, y=None, w_post=None, gate=None, w_pre=None, r=None, h=None,
                      q=None, q_scale=None, stream=None):
    """r = res_scale x + gate norm(y, w_post), h = norm(r, w_pre), and h's 8-bit
    codes q with q_scale; what is None falls out (see the header)."""
    s, dev = shape, _device("x, y", x if y is None else y)
    T_, d, dt = s.T, s.d_model, _DTYPE.get(s.dtype)
    gates = -(-T_ // s.rows_per_gate) * d if gate is not None else 0
    io = MoeNormIO(*_matrix("x", x, dt, T_, d, dev), *_matrix("y", y, dt, T_, d, dev),
                   _opt("w_post", w_post, dt, d, dev), _opt("gate", gate, dt, gates, dev),
                   _opt("w_pre", w_pre, dt, d, dev), *_matrix("r", r, dt, T_, d, dev),
                   *_matrix("h", h, dt, T_, d, dev), _opt("q", q, torch.int8, T_ * d, dev),
                   _opt("q_scale", q_scale, torch.float32, T_, dev))
    _run("moe_norm_residual", dev, stream, ctypes.byref(s), ctypes.byref(io))


def moe_norm_residual_backward_workspace_bytes(shape: MoeNormShape) -> int:
    return int(lib().moe_norm_residual_backward_workspace_bytes(ctypes.byref(shape)))


def moe_norm_residual_backward(shape: MoeNormShape, ws, *, r=None, y=None, w_post=None, gate=None, w_pre=None,
                               dr=None, dh=None, dx=None, dy=None, dgate=None, dw_post=None, dw_pre=None,
                               accumulate=False, stream=None):
    """Gradients of moe_norm_residual from dr and dh, the gradients at r and h;
    r, y and the vectors as the forward pass left and had them."""
    s, dev = shape, _device("ws", ws)
    T_, d, dt = s.T, s.d_model, _DTYPE.get(s.dtype)
    gates = -(-T_ // s.rows_per_gate) * d if gate is not None else 0
    io = MoeNormGradIO(*_matrix("r", r, dt, T_, d, dev), *_matrix("y", y, dt, T_, d, dev),
                       _opt("w_post", w_post, dt, d, dev), _opt("gate", gate, dt, gates, dev),
                       _opt("w_pre", w_pre, dt, d, dev), *_matrix("dr", dr, dt, T_, d, dev),
                       *_matrix("dh", dh, dt, T_, d, dev), *_matrix("dx", dx, dt, T_, d, dev),
                       *_matrix("dy", dy, dt, T_, d, dev), _opt("dgate", dgate, dt, gates, dev),
                       _opt("dw_post", dw_post, dt, d, dev), _opt("dw_pre", dw_pre, dt, d, dev),
                       int(bool(accumulate)), 0)
    _run("moe_norm_residual_backward", dev, stream, ctypes.byref(s), ctypes.byref(io),
         _scratch(ws, _on(dev, moe_norm_residual_backward_workspace_bytes, s), dev))


# ---- a block: selection, experts and the residual step behind them


class I8Experts:
    """The experts' weights in 8 bits: codes and the scales of their output
    channels, laid out once (quantize_rows, on `stream`, to which they belong)."""

    def __init__(self, w_gate, w_up, w_down, stream=None):
        (self.w_gate, self.s_gate), (self.w_up, self.s_up), (self.w_down, self.s_down) = (
            quantize_rows(w, stream) for w in (w_gate, w_up, w_down))


class BlockBuffers:
    """Device buffers of one block: the layer's (binding.LayerBuffers), its
    logits, the new residual r and the next block's input h; with i8, the codes
    of h and the experts' workspace."""

    def __init__(self, shape: B.MoeShape, i8=False, device="cuda"):
        self.shape, self.layer = shape, B.LayerBuffers(shape, device)
        dt, rows = _DTYPE[shape.dtype], (shape.T, shape.d_model)
        self.logits = torch.empty((shape.T, shape.n_ffn + shape.n_zero), dtype=torch.float32, device=device)
        self.r, self.h = torch.empty(rows, dtype=dt, device=device), torch.empty(rows, dtype=dt, device=device)
        self.q = self.q_scale = self.ws = None
        if i8:
            self.q = torch.empty(rows, dtype=torch.int8, device=device)
            self.q_scale = torch.empty(shape.T, dtype=torch.float32, device=device)
            self.ws = torch.empty(moe_expert_ffn_i8_workspace_bytes(shape), dtype=torch.uint8, device=device)


def block_input(norm: MoeNormShape, buf: BlockBuffers, x, w_pre, stream=None):
    """The first block's input, h = x rstd(x) w_pre (and its codes), in ``buf``,
    which stands for the block before it; norm: res_scale 1."""
    moe_norm_residual(norm, x=x, w_pre=w_pre, h=buf.h, q=buf.q, q_scale=buf.q_scale, stream=stream)
    return buf.h


def block_forward(buf: BlockBuffers, params: MoeSelectParams, norm: MoeNormShape, x, before: BlockBuffers, w_router,
                  bias, experts, *, w_post=None, gate=None, w_pre=None, logit_bias=None, stream=None):
    """One block on the residual x and its input before.h: selection, experts
    (I8Experts, or w_gate, w_up, w_down) and combine, then r = res_scale x + gate
    norm(y, w_post) and the next block's input h = norm(r, w_pre), in ``buf``."""
    s, L, h = buf.shape, buf.layer, before.h
    dev = _device("before.h", h)
    if dev != torch.cuda.current_device():      # (the layer's own calls go by the current device)
        with torch.cuda.device(dev):
            return block_forward(buf, params, norm, x, before, w_router, bias, experts, w_post=w_post, gate=gate,
                                 w_pre=w_pre, logit_bias=logit_bias, stream=stream)
    moe_route_select(s, params, h, w_router, logit_bias, bias, L.topk_idx, L.topk_gate, buf.logits, L.ws, stream)
    B.moe_dispatch(s, L.topk_idx, h, L.counts, L.offsets, L.perm, L.inv_perm, L.x_perm, L.ws, stream)
    if isinstance(experts, I8Experts):
        tokens = dict(x=h) if before.q is None else dict(xq=before.q, x_scale=before.q_scale)
        e = experts
        moe_expert_ffn_i8(s, FfnI8IO(perm=L.perm, offsets=L.offsets, w_gate=e.w_gate, s_gate=e.s_gate, w_up=e.w_up,
                                     s_up=e.s_up, w_down=e.w_down, s_down=e.s_down, y_perm=L.y_perm, **tokens),
                          buf.ws, stream)
    else:
        B.moe_expert_ffn(s, h, L.x_perm, L.perm, L.offsets, *experts, L.y_perm, L.ws, stream)
    B.moe_combine(s, h, L.y_perm, L.topk_idx, L.topk_gate, L.inv_perm, L.y, stream)
    out = {} if w_pre is None else dict(h=buf.h, q=buf.q, q_scale=buf.q_scale)
    moe_norm_residual(norm, x=x, y=L.y, w_post=w_post, gate=gate, w_pre=w_pre, r=buf.r, stream=stream, **out)
    return buf.r


class BlockGrads:
    """What the backward pass of a block needs beside its BlockBuffers: the
    layer's gradients (train.TrainBuffers; its dx is the gradient at the block's
    input), those at x and y, of the norms' vectors and the gate, workspace."""

    def __init__(self, shape: B.MoeShape, norm: MoeNormShape, w_post=None, gate=None, w_pre=None, device="cuda"):
        self.layer = T.TrainBuffers(shape, device)
        like = self.layer.dx
        self.dx, self.dy = torch.empty_like(like), torch.empty_like(like)
        self.dw_post, self.dgate, self.dw_pre = (None if t is None else torch.zeros_like(t)
                                                 for t in (w_post, gate, w_pre))
        self.ws = torch.empty(moe_norm_residual_backward_workspace_bytes(norm), dtype=torch.uint8, device=device)


def block_backward(buf: BlockBuffers, g: BlockGrads, params: MoeSelectParams, norm: MoeNormShape, before: BlockBuffers,
                   w_router, experts, dr, dh=None, *, w_post=None, gate=None, w_pre=None, accumulate=False,
                   stream=None):
    """Gradients of the last ``block_forward`` on ``buf`` (experts w_gate, w_up,
    w_down) from those at r and h: at x in ``g.dx``, at the block's input in
    ``g.layer.dx``, which are the block before's dr and dh."""
    moe_norm_residual_backward(norm, g.ws, r=buf.r if w_pre is not None else None, y=buf.layer.y, w_post=w_post,
                               gate=gate, w_pre=w_pre, dr=dr, dh=dh, dx=g.dx, dy=g.dy, dgate=g.dgate,
                               dw_post=g.dw_post, dw_pre=g.dw_pre, accumulate=accumulate, stream=stream)
    L, t = buf.layer, g.layer
    io = T.BackwardIO(x=before.h, w_router=w_router, logits=buf.logits, topk_idx=L.topk_idx, topk_gate=L.topk_gate,
                      offsets=L.offsets, perm=L.perm, inv_perm=L.inv_perm, w_gate=experts[0], w_up=experts[1],
                      w_down=experts[2], dy=g.dy, dx=t.dx, dgate=t.dgate, dlogits=t.dlogits, dw_router=t.dw_router,
                      dw_gate=t.dw_gate, dw_up=t.dw_up, dw_down=t.dw_down, accumulate=accumulate)
    moe_layer_backward_select(buf.shape, params, io, t.ws, stream)
    return g.dx, t.dx
