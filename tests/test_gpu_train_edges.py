"""The training operators at the edges of what moe_train.h allows: more tokens
than a launch has workgroups, a selection that names an expert twice;
the gradient of the logits' offsets, which the caller forms."""

import pytest
import torch

from sparse_moe_layer_03_amd import binding as B
from tests.test_gpu_layer_backward import Case, TOL, far

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_tokens_than_workgroups(dtype):
    # the kernels that have a token or row per workgroup walk over them in
    # strides of 2^20; the second stride is 77 tokens long.  TOL holds: a weight
    # gradient sums 2^17 rows in blocks of 128 (fp32) or runs of 32 (bf16), n
    # additions of up to 2^-23 of the running sum, in the norm sqrt(n / 2) 2^-23
    # with n = 2^10 or 2^12.
    T = (1 << 20) + 77
    say(f"[edges] {dtype} T={T}")
    c = Case(dtype, T, 64, 6, 2, 64, 1, 1.5, 0.5)
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
