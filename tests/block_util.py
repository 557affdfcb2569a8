"""References in 64 bits for the tests of the operators around the layer, and
the bounds that their results are held to."""

import math

import torch

U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step of a rounding
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LEAST = 2.0 ** -126


def say(*a):
    print(*a, flush=True)


# ---- selection


def scores(params, logits):
    """p in 64 bits: 0 for a logit of -inf, also in a row that holds no other."""
    x = logits.double()
    if params.score == 1:
        return torch.sigmoid(x)
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(x - m)
    s = e.sum(1, keepdim=True)
    return e / torch.where(s == 0, torch.ones_like(s), s)


def first(keys, n):
    """The n largest of each row (ties: lowest index), ascending; NaN as -inf."""
    keys = torch.where(torch.isnan(keys), torch.full_like(keys, -math.inf), keys)
    return torch.sort(keys, dim=-1, descending=True, stable=True).indices[..., :n].sort(dim=-1).values


def select_ref(params, logits, bias, top_k, scaling):
    """(idx, gates, p) of the definition in 64 bits."""
    p = scores(params, logits)
    key = p + bias.double() if bias is not None else p
    key = torch.where(torch.isnan(key), torch.full_like(key, -math.inf), key)
    T, E = key.shape
    G = params.n_groups
    if G > 1:
        per = key.view(T, G, E // G)
        top = per.topk(params.group_best, dim=2).values
        best = top[..., 0]
        if params.group_best == 2:      # a second key of -inf does not count
            alone = (best == math.inf) | (top[..., 1] == -math.inf)
            best = torch.where(alone, best, top.sum(2))
        kept = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter_(1, first(best, params.top_groups), True)
        out = (~kept).repeat_interleave(E // G, 1)
        at = torch.sort(key, dim=1, descending=True, stable=True).indices
        at = at.gather(1, torch.sort(out.gather(1, at).to(torch.uint8), dim=1, stable=True).indices)
        idx = at[:, :top_k].sort(dim=1).values
    else:
        idx = first(key, top_k)
    f = p.gather(1, idx)
    if params.renorm:
        d = f.sum(1, keepdim=True) + params.renorm_eps
        f = torch.where(d == 0, torch.zeros_like(f), f / d)
    return idx, scaling * f, p


def select_bwd_ref(params, logits, idx, dgate, scaling):
    """dlogits in 64 bits, and the sum of its terms' magnitudes."""
    p = scores(params, logits)
    E = p.shape[1]
    inside = (idx >= 0) & (idx < E)
    at = torch.where(inside, idx, torch.zeros_like(idx)).long()
    sel = torch.where(inside, p.gather(1, at), torch.zeros_like(dgate, dtype=torch.float64))
    dg = dgate.double()
    d, mag = scaling * dg, (scaling * dg).abs()
    if params.renorm:
        D = sel.sum(1, keepdim=True) + params.renorm_eps
        r = torch.where(D == 0, torch.zeros_like(D), 1 / D)
        d = scaling * r * (dg - (dg * sel).sum(1, keepdim=True) * r)
        mag = abs(scaling) * r * (dg.abs() + (dg.abs() * sel).sum(1, keepdim=True) * r)
    zero = torch.zeros_like(p)
    dp = zero.clone().scatter_add_(1, at, torch.where(inside, d, torch.zeros_like(d)))
    mp = zero.clone().scatter_add_(1, at, torch.where(inside, mag, torch.zeros_like(d)))
    if params.score == 1:
        return p * (1 - p) * dp, p * (1 - p) * mp + p * p * mp
    return p * (dp - (p * dp).sum(1, keepdim=True)), p * (mp + (p * mp).sum(1, keepdim=True))


def score_error(params, logits):
    """Relative error of a score: softmax, exp's argument l - m rounded to 2^-24
    of itself, twice (the score's own and the sum's), up to 40 additions of the
    sum and some 16 roundings of exp, division and products; sigmoid, some 16
    roundings."""
    if params.score == 1:
        return 16 * 2.0 ** -23
    x = logits.double()
    x = torch.where(torch.isfinite(x), x, torch.zeros_like(x))
    span = (x.amax(1, keepdim=True) - x.amin(1, keepdim=True)).clamp(max=88.0)
    return (2 * span + 56) * 2.0 ** -23


# ---- 8-bit integers


def quantise_ref(x):
    """Codes (64-bit floats) and scales (fp32) of rows."""
    top = x.abs().amax(1, keepdim=True).double()
    scale = (top / 127).float().clamp(min=LEAST)
    q = torch.round(x.double() / scale.double())
    bad = ~torch.isfinite(x.double()).all(1, keepdim=True)
    return torch.where(bad, torch.zeros_like(q), q), torch.where(bad, torch.full_like(scale, math.nan), scale)[:, 0]


def matmul_ref(counts, q, sa, w, sw, out_dtype):
    """The product's bits: an exact sum, converted and multiplied in fp32."""
    out, lo = [], 0
    for e, n in enumerate(counts):
        acc = q[lo:lo + n].double() @ w[e].double().t()
        out.append((acc.float() * sa[lo:lo + n, None] * sw[e]).to(out_dtype))
        lo += n
    return torch.cat(out)


def codes(shape, g, low=-127):
    return torch.randint(low, 128, shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int8)


# ---- norms


def rstd(v, eps):
    return 1 / (v.square().mean(1, keepdim=True) + eps).sqrt()


def gate_rows(gate, T, per):
    return gate.double()[torch.arange(T, device=gate.device) // per]
