"""What the operators around the layer may write and read: every array lies
inside a larger buffer of 0xff bytes (NaN in bf16 and fp32, -1 in codes), as in
tests/test_gpu_train_guards.py, and after a call every byte that is not part of
a written element has to be as it was.  What is read outside an array shows as
NaN, or in the exact values of the codes and products."""


import pytest
import torch

from sparse_moe_layer_03_amd import binding as B
from sparse_moe_layer_03_amd import block as K
from tests.block_util import DT, codes, matmul_ref, quantise_ref, say, select_bwd_ref, select_ref
from tests.test_gpu_i8 import Ffn
from tests.test_gpu_train_guards import Guarded
from tests.train_util import offsets_of

pytestmark = pytest.mark.gpu


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def rows(T, d, dt, ld, fill=None):
    return Guarded((T, d), dt, (ld, 1), fill)


@pytest.mark.parametrize("T,E,k,ld,rule", [(1, 1, 1, 1, ("softmax",)), (37, 96, 8, 101, ("softmax",)), (300, 768, 12, 768, ("sigmoid", 8, 4, 2, True)),
                                           (65, 1023, 16, 1030, ("sigmoid", 33, 17, 1, True)), (9, 200, 3, 200, ("softmax", 8, 3, 2, True))])
def test_selection(T, E, k, ld, rule):
    say(f"[guards] select T={T} E={E} k={k} ld={ld} {rule}")
    s, p, g = B.make_shape(T, 64, E, 0, 64, k, "bf16", 1.5), K.make_select(*rule), gen()
    logits = rows(T, E, torch.float32, ld, torch.randn((T, E), generator=g, device="cuda"))
    bias = Guarded((E,), torch.float32, fill=torch.randn(E, generator=g, device="cuda") * 0.01)
    idx, gate = Guarded((T, k), torch.int32), Guarded((T, k), torch.float32)
    dgate = Guarded((T, k), torch.float32, fill=torch.randn((T, k), generator=g, device="cuda"))
    dlogits = Guarded((T, E), torch.float32)
    K.moe_select(s, p, logits.t, bias.t, idx.t, gate.t)
    K.moe_select_backward(s, p, logits.t, idx.t, dgate.t, dlogits.t)
    torch.cuda.synchronize()
    for n, a, w in (("logits", logits, False), ("bias", bias, False), ("idx", idx, True), ("gate", gate, True),
                    ("dgate", dgate, False), ("dlogits", dlogits, True)):
        a.check(n, written=w)
    want, wg, _ = select_ref(p, logits.t, bias.t, k, 1.5)
    assert torch.equal(idx.t.long(), want) and ((gate.t - wg).abs() < 1e-5).all()
    ref, mag = select_bwd_ref(p, logits.t, want, dgate.t, 1.5)
    assert ((dlogits.t - ref).abs() <= 1e-4 * mag + 1e-9).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,Kn,ldx,ldq", [(5, 64, 64, 64), (33, 1001, 1003, 1005), (3, 8, 9, 11), (2, 3, 3, 3), (7, 2056, 2056, 2057),
                                          (2, 40000, 40001, 40000)])
def test_quantize(dtype, M, Kn, ldx, ldq):
    x = rows(M, Kn, DT[dtype], ldx, torch.randn((M, Kn), generator=gen(), device="cuda"))
    q, scale = rows(M, Kn, torch.int8, ldq), Guarded((M,), torch.float32)
    K.moe_quantize_rows(K.make_quant_shape(dtype, M, Kn, ldx, ldq), x.t, q.t, scale.t)
    torch.cuda.synchronize()
    x.check("x", written=False), q.check("q"), scale.check("scale")
    wq, ws = quantise_ref(x.t)
    assert torch.equal(q.t.double(), wq) and torch.equal(scale.t, ws)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("counts,N,Kn,lda,ldc", [((5, 70, 0, 33, 129), 72, 160, 176, 76), ((5, 70, 0, 33, 129), 70, 160, 160, 71),
                                                 ((5, 70, 0, 33, 129), 33, 77, 79, 33), ((1,), 520, 6144, 6144, 520),
                                                 ((3,), 37, 6143, 6145, 39), ((300, 2, 261), 4096, 128, 128, 4096),
                                                 ((200, 90, 130), 4096, 144, 160, 4100), ((40,) * 30, 2048, 128, 128, 2048),
                                                 ((4,) * 40, 2048, 128, 128, 2048)])
def test_products(out, counts, N, Kn, lda, ldc):
    say(f"[guards] matmul_i8 {counts[:5]} N={N} K={Kn} {out}")
    g, G, first, n = gen(), len(counts), 3, sum(counts)
    M = first + n + 6
    s = K.make_i8_shape(out, G, M, N, Kn, lda, ldc)
    a, w = rows(M, Kn, torch.int8, lda), Guarded((G, N, Kn), torch.int8, fill=codes((G, N, Kn), g))
    a.t[first:first + n] = codes((n, Kn), g)
    a.keep()
    sa, sw = Guarded((M,), torch.float32), Guarded((G, N), torch.float32, fill=torch.rand((G, N), generator=g, device="cuda"))
    sa.t[first:first + n] = torch.rand(n, generator=g, device="cuda")
    sa.keep()
    o, ws = rows(M, N, DT[out], ldc), Guarded((K.moe_matmul_i8_workspace_bytes(s),), torch.uint8)
    off = Guarded((G + 1,), torch.int32, fill=offsets_of(list(counts)) + first)
    K.moe_matmul_i8(s, off.t, a.t, sa.t, w.t, sw.t, o.t, ws.t)
    torch.cuda.synchronize()
    for name, v in (("a", a), ("sa", sa), ("w", w), ("sw", sw), ("offsets", off)):
        v.check(name, written=False)
    ws.check("ws")
    o.check("out", (first, first + n))
    part = slice(first, first + n)
    assert torch.equal(o.t[part], matmul_ref(counts, a.t[part], sa.t[part], w.t, sw.t, DT[out]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,n,z,k", [(1, 64, 64, 4, 2, 2), (90, 192, 320, 6, 3, 3), (700, 128, 192, 2, 1, 2)])
def test_ffn(dtype, T, d, f, n, z, k):
    say(f"[guards] ffn_i8 {dtype} T={T}")
    c = Ffn(T, d, f, n, z, k, dtype)
    kept = {name: Guarded(tuple(t.shape), t.dtype, fill=t) for name, t in
            (("x", c.x), ("perm", c.perm), ("offsets", c.offsets), *c.w.items())}
    y, ws = Guarded((T * k, d), c.dt), Guarded((c.ws.numel(),), torch.uint8)
    K.moe_expert_ffn_i8(c.s, K.FfnI8IO(y_perm=y.t, **{name: a.t for name, a in kept.items()}), ws.t)
    torch.cuda.synchronize()
    for name, a in kept.items():
        a.check(name, written=False)
    ws.check("ws")
    used = sum(c.counts[:n])
    y.check("y_perm", (0, used))
    c.y[:used] = y.t[:used]
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,ld,per", [(1, 1, 1, 1), (40, 64, 64, 7), (40, 100, 101, 7), (300, 1003, 1009, 40), (9, 2048, 2050, 2),
                                        (5, 6144, 6144, 5), (3, 9001, 9002, 1)])
def test_norms(dtype, T, d, ld, per):
    say(f"[guards] norm {dtype} T={T} d={d} ld={ld} per={per}")
    g, dt = gen(), DT[dtype]
    s = K.make_norm_shape(T, d, dtype, 1e-6, 0.5, per)
    new = lambda: torch.randn((T, d), generator=g, device="cuda")  # noqa: E731
    vec = lambda *n: Guarded(n, dt, fill=torch.randn(n, generator=g, device="cuda") + 1)  # noqa: E731
    n_gates = -(-T // per)
    ins = {"x": rows(T, d, dt, ld, new()), "y": rows(T, d, dt, ld, new()), "w_post": vec(d), "gate": vec(n_gates, d),
           "w_pre": vec(d)}
    outs = {"r": rows(T, d, dt, ld), "h": rows(T, d, dt, ld), "q": Guarded((T, d), torch.int8),
            "q_scale": Guarded((T,), torch.float32)}
    K.moe_norm_residual(s, **{n: a.t for n, a in (ins | outs).items()})
    torch.cuda.synchronize()
    for n, a in ins.items():
        a.check(n, written=False)
    for n, a in outs.items():
        a.check(n)
        assert torch.isfinite(a.t.float()).all(), n
    wq, wsc = quantise_ref(outs["h"].t)
    assert torch.equal(outs["q"].t.double(), wq) and torch.equal(outs["q_scale"].t, wsc)
    outs["r"].keep()
    back = {"r": outs["r"], **{n: ins[n] for n in ("y", "w_post", "gate", "w_pre")}, "dr": rows(T, d, dt, ld, new()),
            "dh": rows(T, d, dt, ld, new())}
    grads = {"dx": rows(T, d, dt, ld), "dy": rows(T, d, dt, ld), "dgate": Guarded((n_gates, d), dt),
             "dw_post": Guarded((d,), dt), "dw_pre": Guarded((d,), dt)}
    ws = Guarded((K.moe_norm_residual_backward_workspace_bytes(s),), torch.uint8)
    K.moe_norm_residual_backward(s, ws.t, **{n: a.t for n, a in (back | grads).items()})
    torch.cuda.synchronize()
    for n, a in back.items():
        a.check(n, written=False)
    for n, a in grads.items():
        a.check(n)
        assert torch.isfinite(a.t.float()).all(), n
    ws.check("ws")
