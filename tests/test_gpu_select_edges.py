"""Selections and their gradient at the ends of fp32's range, against the
definition in 64 bits."""

import math

import pytest
import torch

from sparse_moe_layer_03_amd import block as K
from tests.block_util import say, score_error, scores, select_ref
from tests.test_gpu_select import check, shape

pytestmark = pytest.mark.gpu
LOW = torch.finfo(torch.float32).min


def logits_of(T, E, seed=0):
    return torch.randn((T, E), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("kept", [1, 2, 3, 4, 5])
def test_groups_switched_off_by_the_types_lowest_value(score, best, kept):
    """Biases of fp32's lowest value add up to more than fp32 holds; such a group
    still comes before one whose experts have -inf."""
    T, E, G = 70, 48, 6
    bias = torch.zeros((G, E // G), device="cuda")
    bias[0] = -math.inf
    bias[1] = LOW
    bias[2] = -1e38
    bias[2, 1] = LOW
    bias[3, 1:] = LOW
    bias[4] = LOW
    bias[4, 3] = -3e38
    k = min(16, kept * E // G)
    check(T, E, k, (score, G, kept, best, True, 0.0), logits=logits_of(T, E), bias=bias.view(-1))
    bias[5] = LOW
    check(T, E, k, (score, G, kept, best, False, 0.0), logits=logits_of(T, E, 1), bias=bias.view(-1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kept", [1, 2, 4])
def test_groups_of_the_largest_biases(score, kept):
    """Sums of two finite keys beyond fp32's largest number, behind a group with an
    infinite one, in their order."""
    T, E, G = 50, 40, 5
    bias = torch.zeros((G, E // G), device="cuda")
    bias[0, :2] = 2e38
    bias[1, :2] = 3e38
    bias[2, :2] = -LOW
    bias[4, 5] = math.inf
    idx, _ = check(T, E, 8, (score, G, kept, 2, True, 0.0), logits=logits_of(T, E, 2), bias=bias.view(-1))
    assert (idx == 37).any(1).all()


@pytest.mark.parametrize("renorm,eps", [(False, 0.0), (True, 0.0), (True, 1e-3)])
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (300, 96, 8), (40, 768, 12)])
def test_gradient_of_saturated_sigmoids(T, E, k, renorm, eps):
    """Each expert's gradient is p (1 - p) dp with 1 - p = 1 / (1 + exp(l)), which for
    logits above 17 is less than the last bit of p: to a relative bound."""
    say(f"[select_backward, saturated] T={T} E={E} k={k} {renorm} {eps}")
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = (torch.rand((T, E), generator=g, device="cuda") - 0.5) * 60
    p = K.make_select("sigmoid", renorm=renorm, renorm_eps=eps)
    idx = select_ref(p, logits, None, k, 2.5)[0]
    dgate = torch.randn((T, k), generator=g, device="cuda")
    out = torch.full((T, E), math.nan, device="cuda")
    K.moe_select_backward(shape(T, E, k, 2.5), p, logits, idx.to(torch.int32), dgate, out)
    torch.cuda.synchronize()
    x, dg = logits.double().gather(1, idx), dgate.double()
    f, rest = torch.sigmoid(x), torch.sigmoid(-x)
    dp, mag = 2.5 * dg, 2.5 * dg.abs()
    if renorm:
        whole = f.sum(1, keepdim=True) + p.renorm_eps
        apart = dg[:, :, None] - dg[:, None, :]
        dp, mag = (2.5 * ((v * f[:, None, :]).sum(2) + p.renorm_eps * d) / whole ** 2
                   for v, d in ((apart, dg), (apart.abs(), dg.abs())))
    ref, bound = (torch.zeros_like(out, dtype=torch.float64).scatter_(1, idx, f * rest * d) for d in (dp, mag))
    # p, 1 - p and the two factors 1 / D each carry a score's error, as does p in every term of the sum
    assert ((out.double() - ref).abs() <= 8 * score_error(p, logits) * bound).all()
    if not renorm:
        assert ((out != 0).sum(1) == k).all()


def tiny_scores(score, T, E, seed):
    """Logits whose scores, but for softmax's first expert, reach from 2^-60 down
    to 1e-260; rows whose scores are 0 in 64 bits as well."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    depth = torch.rand((T, 1), generator=g, device="cuda") * 550 + 42
    logits = -depth - torch.rand((T, E), generator=g, device="cuda") * torch.rand((T, 1), generator=g, device="cuda") * 40
    logits[1] = -math.inf
    logits[2] = -800.0
    logits[3, 4:] = -800.0
    if score == "softmax":
        logits[:, 0] = 0.0
    return logits


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, 1e-20])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(400, 96, 8), (60, 768, 12), (70, 7, 1)])
def test_renormalised_gates_of_scores_below_fp32s_normal_numbers(T, E, k, score, eps):
    bias = None
    if score == "softmax":                  # the experts behind the one that holds all
        bias = torch.zeros(E, device="cuda")
        bias[0] = -math.inf
    logits = tiny_scores(score, T, E, 5)
    _, gate = check(T, E, k, (score, 1, 1, 1, True, eps), logits=logits, bias=bias)
    if eps == 0:
        have = [t for t in range(T) if t not in (1, 2)]
        assert ((gate[have].sum(1) - 2.5).abs() < 1e-5).all() and (gate[1:3] == 0).all()
    if E % 4 == 0:
        check(T, E, k, (score, 4, 3, 2, True, eps), logits=logits, bias=bias)


@pytest.mark.parametrize("eps", [0.0, 1e-44, 1e-30, 1e-20])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(400, 96, 8), (60, 768, 12), (70, 7, 1)])
def test_gradient_of_renormalised_gates_of_scores_below_fp32s_normal_numbers(T, E, k, score, eps):
    """With f_j = p_j / D: p_e dp_e = s f_e (eps / D dg_e + sum_i f_i (dg_e - dg_i)), and
    sum_j p_j dp_j = s sum_i f_i dg_i eps / D."""
    say(f"[select_backward, small scores] T={T} E={E} k={k} {score} {eps}")
    logits = tiny_scores(score, T, E, 6)
    g = torch.Generator(device="cuda").manual_seed(7)
    p = K.make_select(score, renorm=True, renorm_eps=eps)
    first = int(score == "softmax" and E > 7)
    idx = torch.argsort(torch.rand((T, E - first), generator=g, device="cuda"), 1)[:, :k].sort(1).values + first
    if score == "softmax" and k > 1:
        idx[5:9, 0] = 0                     # (with the one that holds all)
    dgate = torch.randn((T, k), generator=g, device="cuda")
    out = torch.full((T, E), math.nan, device="cuda")
    K.moe_select_backward(shape(T, E, k, 2.5), p, logits, idx.to(torch.int32), dgate, out)
    torch.cuda.synchronize()
    s, dg = scores(p, logits), dgate.double()
    f = s.gather(1, idx)
    D = f.sum(1, keepdim=True) + p.renorm_eps
    f = torch.where(D == 0, f, f / D)
    e = torch.where(D == 0, D, p.renorm_eps / D)
    by = torch.sigmoid(-logits.double().gather(1, idx)) if p.score else 1.0
    apart = dg[:, :, None] - dg[:, None, :]
    ref, bound = (torch.zeros_like(s).scatter_(1, idx, 2.5 * by * f * ((v * f[:, None, :]).sum(2) + e * d))
                  for v, d in ((apart, dg), (apart.abs(), dg.abs())))
    if not p.score:
        ref = ref - s * 2.5 * (f * dg).sum(1, keepdim=True) * e
        bound = bound + s * 2.5 * (f * dg.abs()).sum(1, keepdim=True) * e
    # every score's error in its own share, in the others' and in D; what is held as 0 below 2^-126
    assert ((out.double() - ref).abs() <= 8 * score_error(p, logits) * bound + 2.0 ** -120).all()


def test_infinite_logits():
    """A softmax over +inf is NaN throughout and, its keys being equal, takes the
    lowest ids; a sigmoid of +inf is 1."""
    T, E, k = 5, 96, 4
    logits = logits_of(T, E, 4)
    logits[1, 9] = math.inf
    logits[2, 9] = logits[2, 80] = math.inf
    logits[3, 40], logits[3, 41] = math.inf, math.nan
    for renorm in (False, True):
        idx, gate = check(T, E, k, ("softmax", 1, 1, 1, renorm, 0.0), logits=logits, bias=None)
        assert gate[1:4].isnan().all() and (idx[1:4] == torch.arange(k, device="cuda")).all()
        assert torch.isfinite(gate[[0, 4]]).all()
        idx, gate = check(T, E, k, ("sigmoid", 4, 2, 2, renorm, 0.0), logits=logits, bias=None)
        assert (idx[1] == 9).any() and (idx[2] == 9).any() and (idx[2] == 80).any() and (idx[3] == 40).any()
        assert not (idx[3] == 41).any() and torch.isfinite(gate).all()
        if not renorm:
            assert (gate[2][(idx[2] == 9) | (idx[2] == 80)] == 2.5).all()
