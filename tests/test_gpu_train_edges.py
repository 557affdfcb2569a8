"""The training operators at the edges of what moe_train.h allows: more tokens
than a launch has workgroups, a selection that names an expert twice;
the gradient of the logits' offsets, which the caller forms; errors in the
norm, real widths, streams that have a part of the CUs."""

import pytest
import torch

from sparse_moe_layer_03_amd import binding as B
from sparse_moe_layer_03_amd import scmoe
from sparse_moe_layer_03_amd import train as T
from tests.test_gpu_adamw import HYPER, clone, make as make_adamw
from tests.test_gpu_gmm import make, ragged, run
from tests.test_gpu_layer_backward import Case, TOL, far
from tests.train_util import U, gmm_ref, offsets_of

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_tokens_than_workgroups(dtype):
    # the kernels that have a token or row per workgroup hold them in planes of
    # 2^20; the second plane is 77 tokens long.  TOL holds: a weight
    # gradient sums 2^17 rows in blocks of 128 (fp32) or runs of 32 (bf16), n
    # additions of up to 2^-23 of the running sum, in the norm sqrt(n / 2) 2^-23
    # with n = 2^10 or 2^12.
    Tn = (1 << 20) + 77
    say(f"[edges] {dtype} T={Tn}")
    c = Case(dtype, Tn, 64, 6, 2, 64, 1, 1.5, 0.5)
    for n in ("dx", "dgate", "dlogits", "dw_router", "dw_gate", "dw_up", "dw_down"):
        getattr(c.tb, n).fill_(float("nan"))
    tb, ref = c.backward(), c.reference()
    for name, want in ref.items():
        assert far(getattr(tb, name), want) <= TOL[dtype], name
    assert far(tb.dx[-77:], ref["dx"][-77:]) <= TOL[dtype]
    assert torch.isfinite(tb.dgate).all() and torch.isfinite(tb.dlogits).all()
    # dgate of the last tokens by themselves
    x, dy, idx = c.x[-99:].double(), c.dy[-99:].double(), c.buf.topk_idx[-99:, 0].long()
    want = (x * dy).sum(1)
    for e in range(c.n_ffn):
        t = idx == e
        h = torch.nn.functional.silu(x[t] @ c.wg[e].double().t()) * (x[t] @ c.wu[e].double().t())
        want[t] = ((dy[t] @ c.wd[e].double()) * h).sum(1)
    assert far(tb.dgate[-99:, 0], want) <= 1e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [2, 5, 16])
def test_an_expert_twice_in_a_token(dtype, k):
    # a selection by other means than moe_route: FFN and identity experts come up
    # to k times in a token; the gradient at an expert's logit sums its slots
    say(f"[edges] twice {dtype} k={k}")
    c = Case(dtype, 60, 64, 12, 5, 128, k, 1.5, 1.0)
    g = torch.Generator(device="cuda").manual_seed(k)
    idx = torch.randint(0, 17, (60, k), generator=g, device="cuda")
    idx[:20] = torch.randint(0, 3, (20, k), generator=g, device="cuda")
    idx[20:30] = 13
    idx[30:40] = 4
    idx = idx.sort(dim=1).values
    c.buf.topk_idx.copy_(idx)
    c.buf.topk_gate.copy_(c.scaling * torch.softmax(c.tb.logits, 1).gather(1, idx))
    B.moe_dispatch(c.shape, c.buf.topk_idx, c.x, c.buf.counts, c.buf.offsets, c.buf.perm, c.buf.inv_perm, None,
                   c.buf.ws)
    tb, ref = c.backward(), c.reference()
    for name, want in ref.items():
        assert far(getattr(tb, name), want) <= TOL[dtype], name
    p = torch.softmax(tb.logits.double(), 1)
    dp = torch.zeros_like(p).scatter_add_(1, idx, c.scaling * tb.dgate.double())
    want = p * (dp - (p * dp).sum(1, keepdim=True))
    # fp32 from dgate on, sums of k slots and 17 experts: fewer than 32 roundings
    # of 2^-24 of the terms p dp
    assert ((tb.dlogits.double() - want).abs() <= 32 * 2.0 ** -23 * (p * (dp.abs() + (p * dp.abs()).sum(1, keepdim=True)))).all()
    first = tb.dlogits.clone()
    c.backward()
    assert torch.equal(first, tb.dlogits)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_of_the_logits_offsets(dtype):
    # moe_train.h: the sum of dlogits over the tokens.  dlogits are fp32 from end
    # to end whatever the type: 1e-5 as in the test of dlogits itself, measured
    # by the norm of what the differences p (dp - sum p dp) cancel from
    c = Case(dtype, 300, 128, 9, 4, 128, 3, 2.5, 1.0)
    tb = c.backward()
    leaves = [v.detach() for v in c.leaves()]
    lb = c.lb = c.lb.double().requires_grad_()
    c.loss(*leaves).backward()
    p = torch.softmax(tb.logits.double(), 1)
    dp = torch.zeros_like(p).scatter_(1, c.buf.topk_idx.long(), c.scaling * tb.dgate.double())
    room = 1e-5 * (p * dp).norm().item() * 300 ** 0.5
    assert (tb.dlogits.double().sum(0) - lb.grad).norm().item() <= room
    assert lb.grad.norm().item() > 100 * room


@pytest.mark.parametrize("form", ("fwd", "dx", "dw"))
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("split", [False, True])
def test_errors_in_the_norm(form, dtype, out, odd, split):
    # A sum of n products has n additions, each off by at most 2^-23 of the
    # running sum; with products of random signs that grows like the root of the
    # terms so far, and independent errors add up to sqrt(n / 2) 2^-23 of the
    # result in the norm: 4e-6 at n = 2048, where partial sums in bf16 would
    # leave 1e-3.  The result is rounded once (at most U of each value).
    n = 2048
    counts, N, K = ([n - 5, n], 136, 264) if form == "dw" else ([300, 7, 90], n, n)
    if form != "dw":
        N, K = (136, n) if form == "fwd" else (n, 136)
    if split:                               # few tiles: the reduction in ranges
        counts, N, K = ([n, n], 40, 56) if form == "dw" else ([3, 20], min(N, 264), min(K, 264))
        N, K = (N, n) if form == "fwd" else (n, K) if form == "dx" else (N, K)
    N, K = N + odd, K + odd
    say(f"[edges] norm {form} {dtype} {out} {counts} {N} {K}")
    s, lhs, rhs, o = make(form, dtype, counts, N, K, out=out)
    if split:
        assert T.moe_grouped_matmul_workspace_bytes(s) > 0
    run(s, counts, lhs, rhs, o)
    ref, _, longest = gmm_ref(form, counts, lhs, rhs)
    err = far(o, ref)
    say(f"  {err:.2e}")
    assert err <= (longest / 2) ** 0.5 * 2.0 ** -23 + (U[o.dtype] if out == "bf16" else 0.0)


@pytest.mark.parametrize("case", [("bf16", 4096, 2048, 24, 8, 1024, 4, 1.0, 1.0),
                                  ("bf16", 1500, 4096, 12, 6, 1536, 3, 2.5, 2.0),
                                  ("f32", 700, 2048, 6, 3, 1024, 3, 1.0, 1.0)], ids=lambda c: "-".join(map(str, c)))
def test_layers_of_real_widths(case):
    say("[edges]", case)
    c = Case(*case)
    tb, ref = c.backward(), c.reference()
    for name, want in ref.items():
        err = far(getattr(tb, name), want)
        say(f"  {name} {err:.2e}")
        assert err <= TOL[case[0]], (name, err)


@pytest.mark.parametrize("cus", [32, 64])
def test_on_a_part_of_the_cus(cus):
    # tiles and grids go by the CUs that the stream has; the order of every sum
    # does not, so the results are the whole chip's bit for bit
    jobs = []
    for form, dtype, counts, N, K in (
            ("fwd", "bf16", ragged(40, 90), 1112, 264), ("fwd", "bf16", ragged(60, 200), 2056, 328),
            ("dx", "bf16", ragged(48, 80), 264, 2056), ("dx", "bf16", ragged(60, 200), 328, 2056),
            ("dw", "bf16", ragged(40, 50), 776, 1032), ("dw", "bf16", ragged(9, 700), 264, 520),
            ("dw", "bf16", [1999, 2100], 40, 56), ("fwd", "f32", ragged(30, 90), 392, 136),
            ("dx", "f32", ragged(30, 20), 136, 392), ("dw", "f32", ragged(30, 90), 137, 391),
            ("fwd", "bf16", [3, 20], 48, 2056)):
        s, lhs, rhs, out = make(form, dtype, counts, N, K)
        run(s, counts, lhs, rhs, out)
        ws = torch.empty(T.moe_grouped_matmul_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        jobs.append((out.clone(), (s, offsets_of(counts), lhs, rhs, out, ws)))
    layers = [Case("bf16", 600, 256, 12, 6, 192, 4, 1.0, 1.0), Case("f32", 200, 64, 5, 2, 128, 3, 1.0, 1.0)]
    names = ("dx", "dgate", "dlogits", "dw_router", "dw_gate", "dw_up", "dw_down")
    grads = [{n: getattr(c.backward(), n).clone() for n in names} for c in layers]
    ts = make_adamw([300_001, 77], bits=8)
    twin = clone(ts)
    params = T.make_adamw_params(**HYPER, state_bits=8, seed=3)
    T.moe_adamw(params, T.AdamwTensors(ts), T.new_adamw_state())
    ms = scmoe.MaskedStream(scmoe.cu_mask(B.moe_device_cu_count(), 0, cus, "contiguous"))
    try:
        for want, job in jobs:
            job[4].zero_()
            torch.cuda.synchronize()
            T.moe_grouped_matmul(*job, stream=ms.stream)
            torch.cuda.synchronize()
            say(f"[edges] {cus} CUs, {job[0].form} N={job[0].N} K={job[0].K}")
            assert torch.equal(job[4], want), (job[0].form, job[0].N, job[0].K)
        for c, want in zip(layers, grads):
            c.backward(stream=ms.stream)
            for n in names:
                assert torch.equal(getattr(c.tb, n), want[n]), n
        state = T.new_adamw_state()
        tensors = T.AdamwTensors(twin)
        torch.cuda.synchronize()
        T.moe_adamw(params, tensors, state, stream=ms.stream)
        torch.cuda.synchronize()
        for a, b in zip(ts, twin):
            for k in a:
                if isinstance(a[k], torch.Tensor):
                    assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    finally:
        ms.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_saturated_gates(dtype):
    # gate projections of up to some hundred either way, where exp(-z) is infinite
    # or zero: silu and its slope go to z and 1, or to 0, and nothing is NaN.  The
    # slope's sum 1 + z (1 - s) loses no more than |z| 2^-24 for the z of about 10
    # that weigh in it: within TOL.
    c = Case(dtype, 200, 128, 6, 2, 128, 3, 1.0, 0.5)
    c.wg.mul_(100.0)
    c.forward()
    tb, ref = c.backward(), c.reference()
    z = c.x.double() @ c.wg[0].double().t()
    assert z.max() > 200 and z.min() < -200
    for name, want in ref.items():
        got = getattr(tb, name)
        assert torch.isfinite(got).all(), name
        err = far(got, want)
        say(f"  {name} {err:.2e}")
        assert err <= TOL[dtype], (name, err)
