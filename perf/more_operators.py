"""The operators around and beside the layer's own calls, as cases that can be timed and compared.

Three families of ``sparse_moe_layer_03_amd.block``: the router's other selection rules with their
gradient (``select``, ``select_grad``: softmax or sigmoid scores, a balancing bias, groups of experts,
renormalised gates), products in 8-bit integers with a scale for each row and each output channel
(``i8``: a linear map, dense or grouped by expert, of rows that are quantised on the way; ``ffn``: the
experts' SwiGLU FFN made of them), and the norms before and after a block with its gate and the
residual's scale (``norm``, ``norm_grad``).  ``run`` computes them in elementary torch operations in
32 bits, or, with ``own``, through the framework.
"""

import math

import torch

own = False

BF16, F32, F64, I8 = torch.bfloat16, torch.float32, torch.float64, torch.int8
DTYPES = {"bf16": BF16, "f32": F32}
SIZE = {"bf16": 2, "f32": 4}
LEAST = 2.0 ** -126     # smallest scale of a quantised row


def listed():
    return [
        # one decoding step of the large model: 128 tokens over 512 FFN and 256 identity experts
        {"name": "select_decode", "op": "select", "tokens": 128, "experts": 768, "top_k": 12, "score": "softmax",
         "groups": 1, "top_groups": 1, "group_top": 1, "renorm": False, "scaling": 1.0, "off": 0},
        # its prefill batch with sigmoid scores, the best 4 of 8 groups by their two best experts, some
        # experts switched off by their bias
        {"name": "select_groups_prefill", "op": "select", "tokens": 16384, "experts": 768, "top_k": 12,
         "score": "sigmoid", "groups": 8, "top_groups": 4, "group_top": 2, "renorm": True, "scaling": 2.5, "off": 7},
        # the gradient of a training batch of the skewed model's router
        {"name": "select_grad_batch", "op": "select_grad", "tokens": 8192, "experts": 384, "top_k": 8,
         "score": "softmax", "groups": 1, "top_groups": 1, "group_top": 1, "renorm": False, "scaling": 1.0, "off": 0},
        # a small model's, renormalised, in groups, with an odd number of tokens
        {"name": "select_grad_groups", "op": "select_grad", "tokens": 1021, "experts": 96, "top_k": 8,
         "score": "softmax", "groups": 4, "top_groups": 3, "group_top": 1, "renorm": True, "scaling": 2.5, "off": 0},
        # between two blocks of the large model while decoding: latency counts
        {"name": "norm_decode", "op": "norm", "dtype": "bf16", "tokens": 128, "d": 6144, "gate_rows": 128,
         "post": True, "pre": True, "scale": 1.0},
        # the same at prefill, a gate for each sequence of the batch
        {"name": "norm_prefill", "op": "norm", "dtype": "bf16", "tokens": 16384, "d": 6144, "gate_rows": 2048,
         "post": True, "pre": True, "scale": 1.0},
        # the gradient of a training batch of the skewed model
        {"name": "norm_grad_batch", "op": "norm_grad", "dtype": "bf16", "tokens": 8192, "d": 4096, "gate_rows": 8192,
         "post": True, "pre": True, "scale": 0.5},
        # a tiny 32-bit one with odd sizes on every side, a gate for every 17 tokens
        {"name": "norm_grad_f32_odd", "op": "norm_grad", "dtype": "f32", "tokens": 131, "d": 1001, "gate_rows": 17,
         "post": True, "pre": True, "scale": 0.7},
        # a linear map with odd sizes on every side
        {"name": "i8_dense_odd", "op": "i8", "dtype": "bf16", "out": "bf16", "groups": 1, "rows": 389, "spare": 0,
         "n": 1001, "k": 2049, "zipf": 0.0},
        # the down projection of one batch of the small model; rows behind the last expert's belong to
        # identity experts
        {"name": "i8_batch", "op": "i8", "dtype": "bf16", "out": "bf16", "groups": 64, "rows": 21845, "spare": 10923,
         "n": 2048, "k": 1024, "zipf": 0.7},
        # decoding with the large model's experts: every weight is streamed once
        {"name": "ffn_decode", "op": "ffn", "dtype": "bf16", "tokens": 128, "d": 6144, "n_ffn": 512, "n_zero": 256,
         "d_ff": 2048, "top_k": 12, "skew": 0.0},
        # its prefill batch
        {"name": "ffn_prefill", "op": "ffn", "dtype": "bf16", "tokens": 16384, "d": 6144, "n_ffn": 512,
         "n_zero": 256, "d_ff": 2048, "top_k": 12, "skew": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select_grad", "norm", "norm_grad", "i8", "i8", "ffn", "ffn"])
    if op in ("select", "select_grad"):
        groups = rng.choice([1, 1, 2, 4, 8, 12])
        each = _log(rng, 3, 1024 // groups)
        top_groups = rng.randint((groups + 1) // 2, groups)
        top_k = min(_log(rng, 1, 16), top_groups * each)
        return {"op": op, "tokens": _log(rng, 1, 16384), "experts": groups * each, "top_k": top_k,
                "score": rng.choice(["softmax", "sigmoid"]), "groups": groups, "top_groups": top_groups,
                "group_top": rng.choice([1, 2]), "renorm": rng.random() < 0.5, "scaling": rng.choice([1.0, 2.5]),
                "off": rng.choice([0, 0, each // 3])}
    if op in ("norm", "norm_grad"):
        f32 = rng.random() < 0.3
        while True:
            t, d = _log(rng, 1, 16384), _log(rng, 16, 8192)
            if rng.random() < 0.7:
                d = max(8, d // 64 * 64)
            if t * d * (2 if f32 else 1) <= 16384 * 4096:
                break
        post = rng.random() < 0.7
        return {"op": op, "dtype": "f32" if f32 else "bf16", "tokens": t, "d": d,
                "gate_rows": rng.choice([0, 1, t, max(1, t // 7)]), "post": post, "pre": not post or rng.random() < 0.8,
                "scale": rng.choice([1.0, 0.5])}
    if op == "i8":
        while True:
            groups, rows = rng.choice([1, _log(rng, 1, 256)]), _log(rng, 1, 40960)
            n, k = _log(rng, 24, 6144), _log(rng, 24, 6144)
            if rng.random() < 0.7:
                n, k = max(16, n // 16 * 16), max(16, k // 16 * 16)
            if groups * n * k <= 3.2e9 and rows * n * k <= 5e11:
                break
        f32 = rng.random() < 0.2
        return {"op": "i8", "dtype": "f32" if f32 else "bf16", "out": "f32" if f32 or rng.random() < 0.2 else "bf16",
                "groups": groups, "rows": rows, "spare": 0 if groups == 1 else rng.choice([0, rng.randrange(1, 2000)]),
                "n": n, "k": k, "zipf": 0.0 if groups == 1 else rng.choice([0.0, 0.7, 1.2])}
    while True:
        t, d, ff = _log(rng, 1, 16384), 64 * _log(rng, 1, 96), 64 * _log(rng, 1, 32)
        n_ffn, n_zero = _log(rng, 1, 512), rng.choice([0, _log(rng, 1, 256)])
        top_k = min(_log(rng, 1, 12), n_ffn + n_zero)
        if n_ffn * d * ff <= 3.2e9 and t * top_k * d * ff <= 5e11:
            break
    return {"op": "ffn", "dtype": "f32" if rng.random() < 0.2 else "bf16", "tokens": t, "d": d, "n_ffn": n_ffn,
            "n_zero": n_zero, "d_ff": ff, "top_k": top_k, "skew": rng.choice([0.0, 1.0, 2.0])}


def _touched(groups, rows):
    """Experts that hold rows, on average, when `rows` fall on `groups` evenly."""
    return groups * (1.0 - (1.0 - 1.0 / groups) ** rows)


def _gates(c):
    return -(-c["tokens"] // c["gate_rows"]) if c["gate_rows"] else 0


def work(case):
    c = case
    if c["op"] == "select":
        te = c["tokens"] * c["experts"]
        return {"bytes": 4 * te + 4 * c["experts"] + 8 * c["tokens"] * c["top_k"], "flops": 8.0 * te}
    if c["op"] == "select_grad":
        te = c["tokens"] * c["experts"]
        return {"bytes": 8 * te + 8 * c["tokens"] * c["top_k"], "flops": 8.0 * te}
    if c["op"] in ("norm", "norm_grad"):
        es, td = SIZE[c["dtype"]], c["tokens"] * c["d"]
        arrays = 3 + c["pre"]                       # x, y, r and the next block's input
        vectors = c["post"] + c["pre"] + _gates(c)
        if c["op"] == "norm_grad":
            arrays, vectors = 4 + 2 * c["pre"], 2 * vectors     # y, dr, dx, dy; r and dh too
        return {"bytes": (arrays * td + vectors * c["d"]) * es, "flops": (10.0 if c["op"] == "norm" else 20.0) * td}
    if c["op"] == "i8":
        rows, n, k = c["rows"], c["n"], c["k"]
        touched = _touched(c["groups"], rows)
        return {"bytes": rows * k * SIZE[c["dtype"]] + touched * n * (k + 4) + rows * n * SIZE[c["out"]],
                "flops": 2.0 * rows * n * k}
    t, d, ff, n_ffn = c["tokens"], c["d"], c["d_ff"], c["n_ffn"]
    rows = t * c["top_k"] * n_ffn / (n_ffn + c["n_zero"])
    b = (t * d + rows * d) * SIZE[c["dtype"]] + _touched(n_ffn, rows) * (3.0 * d * ff + 4 * (2 * ff + d)) + 4 * rows
    return {"bytes": b, "flops": 6.0 * rows * d * ff}


# ---- inputs


def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std, dtype=F32):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _prepare_select(c, seed):
    g = _gen(seed)
    t, e = c["tokens"], c["experts"]
    s = {"logits": _normal(g, (t, e), 1.0) + _normal(g, (e,), 0.5), "bias": _normal(g, (e,), 0.01)}
    if c["off"]:
        at = torch.randperm(e, generator=_gen(seed, "cpu"))[:c["off"]]
        s["bias"][at.cuda()] = -math.inf
    s["topk_idx"] = torch.zeros((t, c["top_k"]), dtype=torch.int32, device="cuda")
    s["topk_gate"] = torch.zeros((t, c["top_k"]), device="cuda")
    if c["op"] == "select_grad":
        s["topk_idx"].copy_(_choose(c, s["logits"], s["bias"])[0])
        s["dgate"] = _normal(g, (t, c["top_k"]), 1.0)
        s["dlogits"] = torch.zeros((t, e), device="cuda")
    return s


def _prepare_norm(c, seed):
    g = _gen(seed)
    t, d, dt, n = c["tokens"], c["d"], DTYPES[c["dtype"]], _gates(c)
    s = {"y": _normal(g, (t, d), 3.0, dt), "x": _normal(g, (t, d), 1.0, dt),
         "gate": _normal(g, (n, d), 0.3, dt) + 0.5 if n else None,
         "w_post": _normal(g, (d,), 0.2, dt) + 1 if c["post"] else None,
         "w_pre": _normal(g, (d,), 0.2, dt) + 1 if c["pre"] else None}
    if c["op"] == "norm":
        s["r"], s["h"] = torch.zeros_like(s["x"]), torch.zeros_like(s["x"]) if c["pre"] else None
        return s
    # what the forward pass left, and the gradients that come back
    s["r"] = _plain_norm_of({**s, "case": c})[0]
    del s["x"]
    s["dr"] = _normal(g, (t, d), 1.0, dt)
    s["dh"] = _normal(g, (t, d), 1.0, dt) if c["pre"] else None
    for name in ("gate", "w_post", "w_pre"):
        s["d" + name] = None if s[name] is None else torch.zeros_like(s[name])
    s["dx"], s["dy"] = torch.zeros_like(s["y"]), torch.zeros_like(s["y"])
    return s


def _codes(g, groups, n, k):
    """Weights of std k^-1/2 as 8-bit codes and a scale for each output channel."""
    w = torch.empty((groups, n, k), dtype=I8, device="cuda")
    some = max(1, 2 ** 26 // (n * k))
    for e in range(0, groups, some):
        part = w[e:e + some]
        part.copy_(torch.randn(part.shape, generator=g, device="cuda", dtype=BF16).mul_(36).round_().clamp_(-127, 127))
    return w, (torch.rand((groups, n), generator=g, device="cuda") + 0.5) * (k ** -0.5 / 36)


def _prepare_i8(c, seed):
    g, gc = _gen(seed), _gen(seed, "cpu")
    q = torch.arange(1, c["groups"] + 1, dtype=F64).pow(-c["zipf"])
    q = q[torch.randperm(c["groups"], generator=gc)]
    counts = torch.bincount(torch.multinomial(q / q.sum(), c["rows"], replacement=True, generator=gc),
                            minlength=c["groups"])
    m = c["rows"] + c["spare"]
    offsets = torch.zeros(c["groups"] + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    w, scale = _codes(g, c["groups"], c["n"], c["k"])
    return {"counts": counts.tolist(), "offsets": offsets.cuda(), "x": _normal(g, (m, c["k"]), 1.0, DTYPES[c["dtype"]]),
            "w": w, "w_scale": scale, "out": torch.zeros((m, c["n"]), dtype=DTYPES[c["out"]], device="cuda")}


def _prepare_ffn(c, seed):
    g = _gen(seed)
    t, d, ff, n_ffn, k, dt = c["tokens"], c["d"], c["d_ff"], c["n_ffn"], c["top_k"], DTYPES[c["dtype"]]
    e = n_ffn + c["n_zero"]
    s = {"x": _normal(g, (t, d), 1.0, dt)}
    for name, n, kk in (("gate", ff, d), ("up", ff, d), ("down", d, ff)):
        s["w_" + name], s["s_" + name] = _codes(g, n_ffn, n, kk)
    # what the router and the dispatch leave: the tokens' assignments sorted by expert
    score = _normal(g, (t, e), 1.0) + _normal(g, (e,), c["skew"])
    flat = torch.topk(score, k, dim=1).indices.sort(dim=1).values.reshape(-1)
    s["perm"] = torch.sort(flat, stable=True).indices.to(torch.int32)
    counts = torch.bincount(flat, minlength=e)
    s["offsets"] = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    s["offsets"][1:] = counts.cumsum(0)
    s["counts"] = counts[:n_ffn].tolist()
    s["y_perm"] = torch.zeros((t * k, d), dtype=dt, device="cuda")
    return s


def prepare(case, seed):
    make = {"select": _prepare_select, "select_grad": _prepare_select, "norm": _prepare_norm,
            "norm_grad": _prepare_norm, "i8": _prepare_i8, "ffn": _prepare_ffn}[case["op"]]
    return {"case": case, **make(case, seed)}


# ---- the plain forms


def _first(keys, n):
    """The n largest along the last axis, ties to the lowest index, in ascending order of the index."""
    return torch.sort(keys, dim=-1, descending=True, stable=True).indices[..., :n].sort(dim=-1).values


def _choose(c, logits, bias):
    """Selection in 64 bits, since keys may lie next to each other, and the scores of all experts."""
    score = torch.softmax(logits.double(), 1) if c["score"] == "softmax" else torch.sigmoid(logits.double())
    key = score + bias.double()
    if c["groups"] > 1:
        each = c["experts"] // c["groups"]
        per = key.view(-1, c["groups"], each)
        kept = _first(per.topk(c["group_top"], dim=2).values.sum(2), c["top_groups"])
        inside = torch.zeros((key.shape[0], c["groups"]), dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        # experts of the other groups come behind all of the kept ones'
        at = torch.sort(key, dim=1, descending=True, stable=True).indices
        out = (~inside).repeat_interleave(each, 1).gather(1, at)
        idx = at.gather(1, torch.sort(out.to(torch.uint8), dim=1, stable=True).indices[:, :c["top_k"]])
        idx = idx.sort(dim=1).values
    else:
        idx = _first(key, c["top_k"])
    return idx, score


def _plain_select(s):
    c = s["case"]
    idx, _ = _choose(c, s["logits"], s["bias"])
    p = torch.softmax(s["logits"], 1) if c["score"] == "softmax" else torch.sigmoid(s["logits"])
    gate = p.gather(1, idx)
    if c["renorm"]:
        gate = gate / gate.sum(1, keepdim=True)
    s["topk_idx"].copy_(idx)
    s["topk_gate"].copy_(c["scaling"] * gate)
    return {"topk_idx": s["topk_idx"], "topk_gate": s["topk_gate"]}


def _plain_select_grad(s):
    c, idx, dg = s["case"], s["topk_idx"].long(), s["dgate"]
    p = torch.softmax(s["logits"], 1) if c["score"] == "softmax" else torch.sigmoid(s["logits"])
    df = c["scaling"] * dg
    if c["renorm"]:
        sel = p.gather(1, idx)
        whole = sel.sum(1, keepdim=True)
        df = (df - (df * sel / whole).sum(1, keepdim=True)) / whole
    dp = torch.zeros_like(p).scatter_(1, idx, df)
    if c["score"] == "softmax":
        s["dlogits"].copy_(p * (dp - (p * dp).sum(1, keepdim=True)))
    else:
        s["dlogits"].copy_(p * (1 - p) * dp)
    return s["dlogits"]


EPS = 1e-6


def _rstd(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)


def _gate_of(s, f=F32):
    """The gate that every token meets."""
    c = s["case"]
    if s["gate"] is None:
        return 1.0
    return s["gate"].to(f)[torch.arange(c["tokens"], device="cuda") // c["gate_rows"]]


def _plain_norm_of(s):
    c, y = s["case"], s["y"].float()
    n = y * _rstd(y) * s["w_post"].float() if c["post"] else y
    r = (c["scale"] * s["x"].float() + _gate_of(s) * n).to(s["x"].dtype)
    if not c["pre"]:
        return r, None
    v = r.float()
    return r, (v * _rstd(v) * s["w_pre"].float()).to(r.dtype)


def _plain_norm(s):
    r, h = _plain_norm_of(s)
    s["r"].copy_(r)
    if h is None:
        return {"r": s["r"]}
    s["h"].copy_(h)
    return {"r": s["r"], "h": s["h"]}


def _norm_grads(s, f):
    """In type f: the gradients at x, y, the gate and both norms' weights."""
    c, y = s["case"], s["y"].to(f)
    out, dr = {}, s["dr"].to(f)
    if c["pre"]:
        v, dh, w = s["r"].to(f), s["dh"].to(f), s["w_pre"].to(f)
        inv = _rstd(v)
        out["dw_pre"] = (dh * v * inv).sum(0)
        g = dh * w
        dr = dr + inv * (g - v * (g * v).mean(1, keepdim=True) * inv * inv)
    out["dx"] = c["scale"] * dr
    gate = _gate_of(s, f)
    inv = _rstd(y) if c["post"] else 1.0
    n = y * inv
    w = s["w_post"].to(f) if c["post"] else 1.0
    if s["gate"] is not None:
        at = torch.arange(c["tokens"], device="cuda") // c["gate_rows"]
        out["dgate"] = torch.zeros((_gates(c), c["d"]), dtype=f, device="cuda").index_add_(0, at, dr * n * w)
    g = dr * gate
    if c["post"]:
        out["dw_post"] = (g * n).sum(0)
        g = g * w
        g = inv * (g - n * (g * n).mean(1, keepdim=True))
    out["dy"] = g
    return out


def _norm_grad_names(s):
    return [n for n in ("dx", "dy", "dgate", "dw_post", "dw_pre") if s[n] is not None]


def _plain_norm_grad(s):
    got = _norm_grads(s, F32)
    return {n: s[n].copy_(got[n]) for n in _norm_grad_names(s)}


def _quantise(x):
    """Codes of rows and their scales; the quotients in 64 bits, since they may lie next to a border."""
    scale = (x.abs().amax(1, keepdim=True).double() / 127).float().clamp(min=LEAST)
    return torch.round(x.double() / scale.double()).float(), scale


def _product(a, w):
    """Whole numbers: products of 1024 codes stay below 2^24, so that they are exact in 32 bits."""
    n, k = w.shape
    if k <= 1024:
        return (a @ w.float().t())
    return sum((a[:, i:i + 1024] @ w[:, i:i + 1024].float().t()).double() for i in range(0, k, 1024))


def _plain_i8(s):
    c, rows = s["case"], s["case"]["rows"]
    q, scale = _quantise(s["x"][:rows])
    parts = zip(torch.split(q, s["counts"]), torch.split(scale, s["counts"]), s["w"], s["w_scale"])
    s["out"][:rows] = torch.cat([_product(a, w).float() * sa * sw for a, sa, w, sw in parts
                                 if a.shape[0]]).to(s["out"].dtype)
    return s["out"]


def _plain_ffn(s):
    c, rows = s["case"], sum(s["counts"])
    q, scale = _quantise(s["x"])
    tok = s["perm"][:rows].long() // c["top_k"]

    # H's codes hang on its last bits: a 32-bit H is computed in 64 bits
    product, f = (_product, F64) if c["dtype"] == "f32" else ((lambda a, w: a @ w.float().t()), F32)

    def expert(e, at):
        a, sa = q[at], scale[at].to(f)
        z, u = (product(a, s[w][e]).to(f) * sa * s[sc][e] for w, sc in (("w_gate", "s_gate"), ("w_up", "s_up")))
        h, sh = _quantise((z * torch.sigmoid(z) * u).to(s["x"].dtype))
        return (product(h, s["w_down"][e]).float() * sh * s["s_down"][e]).to(s["x"].dtype)

    lo = 0
    for e, n in enumerate(s["counts"]):
        if n:
            s["y_perm"][lo:lo + n] = expert(e, tok[lo:lo + n])
        lo += n
    return s["y_perm"]


# ---- the framework's operators


def _select_of(s):
    from sparse_moe_layer_03_amd import binding as B
    from sparse_moe_layer_03_amd import block as K
    c = s["case"]
    if "shape" not in s:
        s["shape"] = B.make_shape(c["tokens"], 64, c["experts"], 0, 64, c["top_k"], "bf16", c["scaling"])
        s["params"] = K.make_select(c["score"], c["groups"], c["top_groups"], c["group_top"], c["renorm"])
    return K


def _own_select(s):
    K = _select_of(s)
    K.moe_select(s["shape"], s["params"], s["logits"], s["bias"], s["topk_idx"], s["topk_gate"])
    return {"topk_idx": s["topk_idx"], "topk_gate": s["topk_gate"]}


def _own_select_grad(s):
    K = _select_of(s)
    K.moe_select_backward(s["shape"], s["params"], s["logits"], s["topk_idx"], s["dgate"], s["dlogits"])
    return s["dlogits"]


def _norm_shape(s):
    from sparse_moe_layer_03_amd import block as K
    c = s["case"]
    if "shape" not in s:
        s["shape"] = K.make_norm_shape(c["tokens"], c["d"], c["dtype"], EPS, c["scale"], c["gate_rows"] or None)
    return K


def _own_norm(s):
    K = _norm_shape(s)
    K.moe_norm_residual(s["shape"], x=s["x"], y=s["y"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"],
                        r=s["r"], h=s["h"])
    return {"r": s["r"], "h": s["h"]} if s["case"]["pre"] else {"r": s["r"]}


def _own_norm_grad(s):
    K = _norm_shape(s)
    if "ws" not in s:
        s["ws"] = torch.empty(K.moe_norm_residual_backward_workspace_bytes(s["shape"]), dtype=torch.uint8, device="cuda")
    K.moe_norm_residual_backward(s["shape"], s["ws"], r=s["r"], y=s["y"], w_post=s["w_post"], gate=s["gate"],
                                 w_pre=s["w_pre"], dr=s["dr"], dh=s["dh"], dx=s["dx"], dy=s["dy"], dgate=s["dgate"],
                                 dw_post=s["dw_post"], dw_pre=s["dw_pre"])
    return {n: s[n] for n in _norm_grad_names(s)}


def _own_i8(s):
    from sparse_moe_layer_03_amd import block as K
    c = s["case"]
    m = c["rows"] + c["spare"]
    if "shape" not in s:
        s["quant"] = K.make_quant_shape(c["dtype"], m, c["k"])
        s["shape"] = K.make_i8_shape(c["out"], c["groups"], m, c["n"], c["k"])
        s["q"] = torch.empty((m, c["k"]), dtype=I8, device="cuda")
        s["q_scale"] = torch.empty(m, device="cuda")
        s["ws"] = torch.empty(K.moe_matmul_i8_workspace_bytes(s["shape"]), dtype=torch.uint8, device="cuda")
    K.moe_quantize_rows(s["quant"], s["x"], s["q"], s["q_scale"])
    K.moe_matmul_i8(s["shape"], s["offsets"], s["q"], s["q_scale"], s["w"], s["w_scale"], s["out"], s["ws"])
    return s["out"]


def _own_ffn(s):
    from sparse_moe_layer_03_amd import binding as B
    from sparse_moe_layer_03_amd import block as K
    c = s["case"]
    if "io" not in s:
        s["shape"] = B.make_shape(c["tokens"], c["d"], c["n_ffn"], c["n_zero"], c["d_ff"], c["top_k"], c["dtype"])
        s["io"] = K.FfnI8IO(**{n: s[n] for n in ("x", "perm", "offsets", "w_gate", "s_gate", "w_up", "s_up", "w_down",
                                                 "s_down", "y_perm")})
        s["ws"] = torch.empty(K.moe_expert_ffn_i8_workspace_bytes(s["shape"]), dtype=torch.uint8, device="cuda")
    K.moe_expert_ffn_i8(s["shape"], s["io"], s["ws"])
    return s["y_perm"]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"select": _own_select, "select_grad": _own_select_grad, "norm": _own_norm, "norm_grad": _own_norm_grad,
                "i8": _own_i8, "ffn": _own_ffn}[op](state)
    return {"select": _plain_select, "select_grad": _plain_select_grad, "norm": _plain_norm,
            "norm_grad": _plain_norm_grad, "i8": _plain_i8, "ffn": _plain_ffn}[op](state)


# ---- the definitions in 64 bits


def _exact_scores(c, s):
    x = s["logits"].double()
    if c["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _exact_select(c, s):
    """One expert after another: the largest key that is left, the lowest id among equals."""
    p = _exact_scores(c, s)
    key = p + s["bias"].double()
    t, each = c["tokens"], c["experts"] // c["groups"]
    rows = torch.arange(t, device="cuda")

    def take(keys, n):
        left, at = torch.ones_like(keys, dtype=torch.bool), []
        ids = torch.arange(keys.shape[1], device="cuda")
        for _ in range(n):
            best = torch.where(left, keys, -math.inf).amax(1, keepdim=True)
            at.append(torch.where(left & (keys == best), ids, keys.shape[1]).amin(1))
            left[rows, at[-1]] = False
        return torch.stack(at, 1)

    if c["groups"] > 1:
        per = key.view(t, c["groups"], each)
        best = per.amax(2)
        if c["group_top"] == 2:
            rest = per.clone()
            rest.scatter_(2, per.argmax(2, keepdim=True), -math.inf)
            best = best + rest.amax(2)
        kept = torch.zeros((t, c["groups"]), dtype=torch.bool, device="cuda")
        kept[rows[:, None], take(best, c["top_groups"])] = True
        # below every key of the kept groups, -inf (an expert that is off) among them
        key = torch.where(key == -math.inf, -1e300, key)
        key = torch.where(kept.repeat_interleave(each, 1), key, -math.inf)
    idx = take(key, c["top_k"]).sort(dim=1).values
    gate = p.gather(1, idx)
    if c["renorm"]:
        gate = gate / gate.sum(1, keepdim=True)
    return {"topk_idx": idx.to(torch.int32), "topk_gate": c["scaling"] * gate}


def _exact_select_grad(c, s):
    """By differentiating the definition."""
    x = s["logits"].double().requires_grad_()
    p = _exact_scores(c, {"logits": x})
    gate = p.gather(1, s["topk_idx"].long())
    if c["renorm"]:
        gate = gate / gate.sum(1, keepdim=True)
    (c["scaling"] * gate).backward(s["dgate"].double())
    return x.grad


def _exact_norm(c, s):
    def norm(v, w):
        return v / (v.pow(2).sum(1, keepdim=True) / c["d"] + EPS).sqrt() * w.double()

    y = s["y"].double()
    r = s["x"].double() * c["scale"]
    n = norm(y, s["w_post"]) if c["post"] else y
    if s["gate"] is not None:
        n = n * s["gate"].double().repeat_interleave(c["gate_rows"], 0)[:c["tokens"]]
    r = r + n
    # the next block reads the sum as it is stored
    return {"r": r, "h": norm(r.to(s["x"].dtype).double(), s["w_pre"])} if c["pre"] else {"r": r}


def _exact_norm_grad(c, s):
    """By differentiating the definition, the stored sum's rounding aside."""
    leaf = {n: s[n].double().requires_grad_() for n in ("y", "r", "gate", "w_post", "w_pre") if s[n] is not None}

    def norm(v, w):
        return v / (v.pow(2).sum(1, keepdim=True) / c["d"] + EPS).sqrt() * w

    dr = s["dr"].double()
    if c["pre"]:
        norm(leaf["r"], leaf["w_pre"]).backward(s["dh"].double())
        dr = dr + leaf["r"].grad
    n = norm(leaf["y"], leaf["w_post"]) if c["post"] else leaf["y"] * 1.0
    if s["gate"] is not None:
        n = n * leaf["gate"].repeat_interleave(c["gate_rows"], 0)[:c["tokens"]]
    n.backward(dr)
    got = {"dx": c["scale"] * dr, "dy": leaf["y"].grad,
           **{"d" + n: leaf[n].grad for n in ("gate", "w_post", "w_pre") if n in leaf}}
    return {n: got[n] for n in _norm_grad_names(s)}


def _exact_quantise(x):
    """Codes and scales in 64 bits; a scale is held in 32."""
    scale = torch.clamp(x.double().abs().amax(1, keepdim=True) / 127, min=LEAST).float().double()
    return torch.round(x.double() / scale), scale


def _exact_i8(c, s):
    out, bounds = s["out"].double(), s["offsets"].tolist()
    for e in range(c["groups"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi > lo:
            q, sa = _exact_quantise(s["x"][lo:hi])
            out[lo:hi] = (q @ s["w"][e].double().t()) * sa * s["w_scale"][e].double()
    return out


def _exact_ffn(c, s):
    out, bounds = s["y_perm"].double(), s["offsets"].tolist()
    tok = torch.div(s["perm"], c["top_k"], rounding_mode="floor").long()
    for e in range(c["n_ffn"]):
        lo, hi = bounds[e], bounds[e + 1]
        if hi == lo:
            continue
        q, sa = _exact_quantise(s["x"][tok[lo:hi]])
        z = (q @ s["w_gate"][e].double().t()) * sa * s["s_gate"][e].double()
        u = (q @ s["w_up"][e].double().t()) * sa * s["s_up"][e].double()
        # H is held in the layer's type before it is quantised
        hq, sh = _exact_quantise((z / (1 + torch.exp(-z)) * u).to(s["x"].dtype))
        out[lo:hi] = (hq @ s["w_down"][e].double().t()) * sh * s["s_down"][e].double()
    return out


def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return {"select": _exact_select, "select_grad": _exact_select_grad, "norm": _exact_norm,
            "norm_grad": _exact_norm_grad, "i8": _exact_i8, "ffn": _exact_ffn}[c["op"]](c, s)
