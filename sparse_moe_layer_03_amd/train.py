"""ctypes binding of the training operators (include/moe_train.h).

Each ``moe_*`` function has the name of the C entry point it calls and takes
torch tensors.  The library checks sizes and alignment; the binding checks
what only it can see: that every tensor lies on one GPU, is laid out as the
call reads it, and is as large as the shape says.  Calls run on the tensors'
device, on its current stream unless ``stream`` names another.
``layer_backward`` and ``train_step`` put the operators together as one
training step of the layer uses them.
"""

from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as B

FORMS = {"fwd": 0, "dx": 1, "dw": 2}
MOE_GMM_FWD, MOE_GMM_DX, MOE_GMM_DW = 0, 1, 2
Q_BLOCK = 256           # elements that share a scale of an 8-bit state
_DTYPE = {B.MOE_F32: torch.float32, B.MOE_BF16: torch.bfloat16}

# every entry point declared in include/moe_train.h
ENTRY_POINTS = ("moe_grouped_matmul_workspace_bytes", "moe_grouped_matmul",
                "moe_layer_backward_workspace_bytes", "moe_layer_backward", "moe_adamw")


class MoeGmmShape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("form", "dtype", "out_dtype", "accumulate", "n_groups",
                                              "M", "N", "K")] + \
               [("lda", ctypes.c_int64), ("ldc", ctypes.c_int64)]


_IO_IN = ("x", "w_router", "logits", "topk_idx", "topk_gate", "offsets", "perm", "inv_perm", "w_gate",
          "w_up", "w_down", "dy")
_IO_OUT = ("dx", "dgate", "dlogits", "dw_router", "dw_gate", "dw_up", "dw_down")


class MoeBackwardIO(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _IO_IN + _IO_OUT] + \
               [("accumulate", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoeAdamwParams(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("state_bits", ctypes.c_int32), ("seed", ctypes.c_uint32)]


class MoeAdamwTensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "master", "m", "v", "m_scale",
                                               "v_scale")] + \
               [("n", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("weight_decay", ctypes.c_double)]


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        L = B.lib()
        vp = ctypes.c_void_p
        L.moe_grouped_matmul_workspace_bytes.argtypes = [ctypes.POINTER(MoeGmmShape)]
        L.moe_grouped_matmul_workspace_bytes.restype = ctypes.c_size_t
        L.moe_grouped_matmul.argtypes = [ctypes.POINTER(MoeGmmShape)] + [vp] * 6
        L.moe_grouped_matmul.restype = ctypes.c_int
        L.moe_layer_backward_workspace_bytes.argtypes = [ctypes.POINTER(B.MoeShape)]
        L.moe_layer_backward_workspace_bytes.restype = ctypes.c_size_t
        L.moe_layer_backward.argtypes = [ctypes.POINTER(B.MoeShape), ctypes.POINTER(MoeBackwardIO),
                                         vp, vp]
        L.moe_layer_backward.restype = ctypes.c_int
        L.moe_adamw.argtypes = [ctypes.POINTER(MoeAdamwParams), ctypes.POINTER(MoeAdamwTensor),
                                ctypes.c_int32, vp, vp, vp, vp]
        L.moe_adamw.restype = ctypes.c_int
        _lib = L
    return _lib


def _dtype_code(dtype) -> int:
    if dtype in ("bf16", torch.bfloat16, B.MOE_BF16):
        return B.MOE_BF16
    if dtype in ("f32", torch.float32, B.MOE_F32):
        return B.MOE_F32
    raise ValueError(f"dtype {dtype}: bf16 or f32")


def _need(name, t, dtype, numel, device=None):
    """t is a contiguous GPU tensor of dtype with at least numel elements."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: a tensor is needed")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name}: on {t.device}, needed on {device or 'a GPU'}")
    if t.dtype != dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise ValueError(f"{name}: {t.dtype}, needed {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, needed {numel}")


def _rows(name, t, dtype, rows, width, ld, device):
    """t holds `rows` rows of `width` elements, `ld` elements apart."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name}: a tensor on {device} is needed")
    if t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, needed {dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] < rows or shape[1] != width or \
            (width > 1 and stride[1] != 1) or (shape[0] > 1 and stride[0] != ld):
        raise ValueError(f"{name}: shape {tuple(shape)} strides {stride}, needed "
                         f"[{rows}, {width}] with strides ({ld}, 1)")


def _workspace(ws, need, device):
    if need and (ws is None or ws.device != device or not ws.is_contiguous()
                 or ws.numel() * ws.element_size() < need):
        raise ValueError(f"ws: {need} bytes on {device} are needed")


def _on(device, call, stream):
    """call(stream's handle) with `device` as the current one; the stream is
    the device's current one by default."""
    if isinstance(stream, torch.cuda.Stream) and stream.device != device:
        raise ValueError(f"stream: on {stream.device}, needed on {device}")
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return call(B._stream(stream))
    return call(B._stream(stream))


# ---- grouped products


def make_gmm_shape(form, dtype, n_groups, M, N, K, out_dtype=None, accumulate=False, lda=None,
                   ldc=None) -> MoeGmmShape:
    """form: "fwd", "dx" or "dw"; lda, ldc: elements between rows of a [M, K]
    and c [M, N] (default: contiguous)."""
    form = FORMS.get(form, form)
    return MoeGmmShape(form, _dtype_code(dtype), _dtype_code(dtype if out_dtype is None else out_dtype),
                       int(bool(accumulate)), n_groups, M, N, K, K if lda is None else lda,
                       N if ldc is None else ldc)


def moe_grouped_matmul_workspace_bytes(shape: MoeGmmShape) -> int:
    return int(lib().moe_grouped_matmul_workspace_bytes(ctypes.byref(shape)))


def moe_grouped_matmul(shape: MoeGmmShape, offsets, lhs, rhs, out, ws=None, stream=None):
    """fwd: out[p] = lhs[p] W_e^T; dx: out[p] = lhs[p] W_e; dw: out[e] = sum
    over the rows p of e of lhs[p]^T rhs[p] (W = rhs, or out)."""
    s = shape
    _need("offsets", offsets, torch.int32, s.n_groups + 1)
    dev, form, M, N, K = offsets.device, s.form, s.M, s.N, s.K
    if s.dtype in _DTYPE and s.out_dtype in _DTYPE and form in (0, 1, 2):
        dt, od, nk = _DTYPE[s.dtype], _DTYPE[s.out_dtype], s.n_groups * N * K
        if form == MOE_GMM_FWD:
            _rows("lhs", lhs, dt, M, K, s.lda, dev)
            _need("rhs", rhs, dt, nk, dev)
            _rows("out", out, od, M, N, s.ldc, dev)
        elif form == MOE_GMM_DX:
            _rows("lhs", lhs, dt, M, N, s.ldc, dev)
            _need("rhs", rhs, dt, nk, dev)
            _rows("out", out, od, M, K, s.lda, dev)
        else:
            _rows("lhs", lhs, dt, M, N, s.ldc, dev)
            _rows("rhs", rhs, dt, M, K, s.lda, dev)
            _need("out", out, od, nk, dev)

    def call(st):
        _workspace(ws, moe_grouped_matmul_workspace_bytes(s), dev)
        return lib().moe_grouped_matmul(ctypes.byref(s), B._p(offsets), B._p(lhs), B._p(rhs),
                                        B._p(out), B._p(ws), st)

    B._check("moe_grouped_matmul", _on(dev, call, stream))


# ---- the layer's backward pass


class BackwardIO:
    """The arrays of one backward pass; keeps its tensors alive.  dlogits, or
    the whole router (w_router, logits, dw_router), may be None."""

    def __init__(self, *, x, w_router, logits, topk_idx, topk_gate, offsets, perm, inv_perm, w_gate,
                 w_up, w_down, dy, dx, dgate, dlogits, dw_router, dw_gate, dw_up, dw_down,
                 accumulate=False):
        given = locals()
        self.tensors = {n: given[n] for n in _IO_IN + _IO_OUT}
        self.accumulate = bool(accumulate)
        self.c = MoeBackwardIO(*[B._p(self.tensors[n]) for n in _IO_IN + _IO_OUT],
                               int(self.accumulate), 0)

    def check(self, s: B.MoeShape):
        t, E, f32, i32 = self.tensors, s.n_ffn + s.n_zero, torch.float32, torch.int32
        dt, Tk, w = _DTYPE.get(s.dtype), s.T * s.top_k, s.n_ffn * s.d_ff * s.d_model
        if dt is None:
            return
        dev = t["x"].device if isinstance(t["x"], torch.Tensor) else None
        need = dict(x=(dt, s.T * s.d_model), dy=(dt, s.T * s.d_model), dx=(dt, s.T * s.d_model),
                    w_router=(dt, E * s.d_model), dw_router=(dt, E * s.d_model),
                    logits=(f32, s.T * E), dlogits=(f32, s.T * E), topk_idx=(i32, Tk),
                    topk_gate=(f32, Tk), dgate=(f32, Tk), offsets=(i32, E + 1), perm=(i32, Tk),
                    inv_perm=(i32, Tk), w_gate=(dt, w), w_up=(dt, w), w_down=(dt, w),
                    dw_gate=(dt, w), dw_up=(dt, w), dw_down=(dt, w))
        for n, (d, k) in need.items():
            if t[n] is None and n in ("w_router", "logits", "dlogits", "dw_router"):
                continue
            _need(n, t[n], d, k, dev)


def moe_layer_backward_workspace_bytes(shape: B.MoeShape) -> int:
    return int(lib().moe_layer_backward_workspace_bytes(ctypes.byref(shape)))


def moe_layer_backward(shape: B.MoeShape, io: BackwardIO, ws, stream=None):
    io.check(shape)
    dev = io.tensors["x"].device

    def call(st):
        _workspace(ws, moe_layer_backward_workspace_bytes(shape), dev)
        return lib().moe_layer_backward(ctypes.byref(shape), ctypes.byref(io.c), B._p(ws), st)

    B._check("moe_layer_backward", _on(dev, call, stream))


# ---- AdamW


def make_adamw_params(lr, beta1=0.9, beta2=0.999, eps=1e-8, state_bits=32, seed=0) -> MoeAdamwParams:
    return MoeAdamwParams(lr, beta1, beta2, eps, state_bits, seed)


class AdamwTensors:
    """The list of parameter tensors of one optimizer.  Each entry is a dict
    with param, grad, m, v, and where used master, m_scale, v_scale and
    weight_decay (default 0).  Arrays that are written may not overlap any
    other (a tied weight is listed once); gradients may overlap each other, and
    an fp32 param may be its own master."""

    def __init__(self, tensors):
        self.tensors = [dict(t) for t in tensors]
        if not self.tensors:
            raise ValueError("no tensors")
        self.device = self.tensors[0]["param"].device
        self.state_bits = 32 if self.tensors[0]["m"].dtype == torch.float32 else 8
        self.c = (MoeAdamwTensor * len(self.tensors))()
        spans = []              # bytes from, to, name, written
        codes = (torch.float8_e4m3fn, torch.uint8)
        for i, t in enumerate(self.tensors):
            n, f32 = t["param"].numel(), torch.float32
            blocks = -(-n // Q_BLOCK)
            kinds = dict(param=tuple(_DTYPE.values()), grad=tuple(_DTYPE.values()))
            if self.state_bits == 32:
                kinds.update(m=f32, v=f32)
            else:
                kinds.update(m=codes, v=codes, m_scale=f32, v_scale=f32)
            if t.get("master") is not None:
                kinds["master"] = f32
            for name, dt in kinds.items():
                held = blocks if name.endswith("_scale") else n
                _need(f"tensors[{i}].{name}", t.get(name), dt, held, self.device)
                at = t[name].data_ptr()
                own = name == "master" and t["param"].dtype == f32 and at == t["param"].data_ptr()
                if held and not own:
                    spans.append((at, at + held * t[name].element_size(), f"tensors[{i}].{name}",
                                  name != "grad"))
            if t["grad"].numel() != n:
                raise ValueError(f"tensors[{i}].grad: {t['grad'].numel()} elements, needed {n}")
            self.c[i] = MoeAdamwTensor(
                *[B._p(t.get(k)) for k in ("param", "grad", "master", "m", "v", "m_scale", "v_scale")],
                n, _dtype_code(t["param"].dtype), _dtype_code(t["grad"].dtype),
                float(t.get("weight_decay", 0.0)))
        spans.sort(key=lambda x: x[:2])
        last = written = (0, 0, "", False)      # of the spans so far, those that end last
        for span in spans:
            other = last if span[3] else written
            if span[0] < other[1]:
                raise ValueError(f"{other[2]} and {span[2]} overlap")
            last = max(last, span, key=lambda x: x[1])
            if span[3]:
                written = max(written, span, key=lambda x: x[1])


def new_adamw_state(device="cuda") -> torch.Tensor:
    """moe_adamw_state as int32[4]: steps taken, steps skipped, 0, 0."""
    return torch.zeros(4, dtype=torch.int32, device=device)


def moe_adamw(params: MoeAdamwParams, tensors: AdamwTensors, state, grad_scale=None, lr_scale=None,
              stream=None):
    if params.state_bits != tensors.state_bits:
        raise ValueError(f"state_bits {params.state_bits}, the tensors' moments have "
                         f"{tensors.state_bits}")
    dev = tensors.device
    _need("state", state, torch.int32, 4, dev)
    for name, t in (("grad_scale", grad_scale), ("lr_scale", lr_scale)):
        if t is not None:
            _need(name, t, torch.float32, 1, dev)
    B._check("moe_adamw", _on(dev, lambda st: lib().moe_adamw(
        ctypes.byref(params), tensors.c, len(tensors.tensors), B._p(state), B._p(grad_scale),
        B._p(lr_scale), st), stream))


# ---- a training step of the layer


class TrainBuffers:
    """What the backward pass of one layer shape needs beside the forward
    pass's LayerBuffers: logits, gradients and workspace."""

    def __init__(self, shape: B.MoeShape, device="cuda"):
        E, dt = shape.n_ffn + shape.n_zero, _DTYPE[shape.dtype]
        new = dict(dtype=dt, device=device)
        f32 = dict(dtype=torch.float32, device=device)
        up = (shape.n_ffn, shape.d_ff, shape.d_model)
        self.logits = torch.empty((shape.T, E), **f32)
        self.dlogits = torch.empty((shape.T, E), **f32)
        self.dgate = torch.empty((shape.T, shape.top_k), **f32)
        self.dx = torch.empty((shape.T, shape.d_model), **new)
        self.dw_router = torch.zeros((E, shape.d_model), **new)
        self.dw_gate, self.dw_up = torch.zeros(up, **new), torch.zeros(up, **new)
        self.dw_down = torch.zeros((shape.n_ffn, shape.d_model, shape.d_ff), **new)
        self.ws = torch.empty(moe_layer_backward_workspace_bytes(shape), dtype=torch.uint8,
                              device=device)


def layer_backward(buf: B.LayerBuffers, tb: TrainBuffers, x, w_router, w_gate, w_up, w_down, dy,
                   accumulate=False, stream=None):
    """Gradients of the last ``binding.layer_forward`` on ``buf``, which was
    given ``tb.logits`` as logits_out; they land in ``tb``."""
    io = BackwardIO(x=x, w_router=w_router, logits=tb.logits, topk_idx=buf.topk_idx,
                    topk_gate=buf.topk_gate, offsets=buf.offsets, perm=buf.perm,
                    inv_perm=buf.inv_perm, w_gate=w_gate, w_up=w_up, w_down=w_down, dy=dy, dx=tb.dx,
                    dgate=tb.dgate, dlogits=tb.dlogits, dw_router=tb.dw_router, dw_gate=tb.dw_gate,
                    dw_up=tb.dw_up, dw_down=tb.dw_down, accumulate=accumulate)
    moe_layer_backward(buf.shape, io, tb.ws, stream)
    return tb.dx


def train_step(buf: B.LayerBuffers, tb: TrainBuffers, x, w_router, bias, w_gate, w_up, w_down,
               loss_grad, params: MoeAdamwParams, tensors: AdamwTensors, state, logit_bias=None,
               grad_scale: Optional[torch.Tensor] = None):
    """Forward, backward and AdamW step of one layer: dy = loss_grad(y).  On
    the current stream, where loss_grad's own work runs too.  The step updates
    what ``tensors`` lists; a logit_bias that is trained has the gradient
    ``tb.dlogits.sum(0)``, which the step does not form."""
    y = B.layer_forward(buf, x, w_router, bias, w_gate, w_up, w_down, logit_bias=logit_bias,
                        logits_out=tb.logits)
    dx = layer_backward(buf, tb, x, w_router, w_gate, w_up, w_down, loss_grad(y))
    moe_adamw(params, tensors, state, grad_scale=grad_scale)
    return y, dx
