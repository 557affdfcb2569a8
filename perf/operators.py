"""The training operators of the MoE layer, as cases that can be timed and compared.

Three operators: the matrix products grouped by expert in the three forms that training needs
(``gmm``: forward, gradient of the rows, gradient of the weights), the backward pass of the whole
layer that is made of them (``layer``), and the AdamW step that applies the gradients (``adamw``).
``run`` computes them in elementary torch operations in 32 bits, or, with ``own``, through
``sparse_moe_layer_03_amd.train``.
"""

import math

import torch

own = False

BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
DTYPES = {"bf16": BF16, "f32": F32}
SIZE = {"bf16": 2, "f32": 4}
Q_BLOCK = 256     # elements that share one scale of an 8-bit state
Q_MAX = 448.0     # largest e4m3 value
MASK32 = 0xFFFFFFFF


def listed():
    return [
        # decoding with the small model's up projection: a few rows per expert, weights streamed once
        {"name": "gmm_fwd_few_rows", "op": "gmm", "form": "fwd", "dtype": "bf16", "out": "bf16",
         "groups": 64, "rows": 389, "spare": 123, "n": 1024, "k": 2048, "zipf": 0.0, "accumulate": False},
        # the down projection of one training batch of the small model; rows behind the last expert's
        # belong to identity experts
        {"name": "gmm_fwd_batch", "op": "gmm", "form": "fwd", "dtype": "bf16", "out": "bf16",
         "groups": 64, "rows": 21845, "spare": 10923, "n": 2048, "k": 1024, "zipf": 0.0, "accumulate": False},
        # gradient of the rows with hot experts: the skewed model's gate projection
        {"name": "gmm_dx_skewed", "op": "gmm", "form": "dx", "dtype": "bf16", "out": "bf16",
         "groups": 256, "rows": 40961, "spare": 0, "n": 1536, "k": 4096, "zipf": 1.2, "accumulate": False},
        # gradient of the weights, summed over micro-batches in 32 bits
        {"name": "gmm_dw_accumulate", "op": "gmm", "form": "dw", "dtype": "bf16", "out": "f32",
         "groups": 64, "rows": 21845, "spare": 77, "n": 1024, "k": 2048, "zipf": 0.0, "accumulate": True},
        # gradient of the weights with ragged experts, many of them short
        {"name": "gmm_dw_ragged", "op": "gmm", "form": "dw", "dtype": "bf16", "out": "bf16",
         "groups": 256, "rows": 10007, "spare": 0, "n": 1536, "k": 4096, "zipf": 1.2, "accumulate": False},
        # a small 32-bit layer with odd sizes on every side
        {"name": "gmm_dx_f32_odd", "op": "gmm", "form": "dx", "dtype": "f32", "out": "f32",
         "groups": 8, "rows": 131, "spare": 5, "n": 251, "k": 129, "zipf": 0.7, "accumulate": False},
        # one step over a model's small tensors (norms, router biases and offsets): launches count
        {"name": "adamw_32_many_small", "op": "adamw", "bits": 32, "tensors": 96, "total": 150001,
         "dtype": "f32", "grad": "f32", "master": False, "decay": 0.0},
        # the small model's experts: weights in bf16 with a 32-bit copy, states in 32 bits
        {"name": "adamw_32_experts", "op": "adamw", "bits": 32, "tensors": 3, "total": 402653184,
         "dtype": "bf16", "grad": "bf16", "master": True, "decay": 0.1},
        # the same with both states in 8 bits
        {"name": "adamw_8_experts", "op": "adamw", "bits": 8, "tensors": 3, "total": 402653184,
         "dtype": "bf16", "grad": "bf16", "master": True, "decay": 0.1},
        # the tiny 32-bit layer: every launch counts
        {"name": "layer_tiny_f32", "op": "layer", "dtype": "f32", "tokens": 64, "d_model": 128, "n_ffn": 8,
         "n_zero": 4, "d_ff": 256, "top_k": 2, "scaling": 1.0, "skew": 0.0, "accumulate": False},
        # one training batch of the small model
        {"name": "layer_small_bf16", "op": "layer", "dtype": "bf16", "tokens": 4096, "d_model": 2048, "n_ffn": 64,
         "n_zero": 32, "d_ff": 1024, "top_k": 8, "scaling": 1.0, "skew": 0.0, "accumulate": False},
        # one training batch of the skewed model: a few hot experts, some with no rows at all
        {"name": "layer_skewed_bf16", "op": "layer", "dtype": "bf16", "tokens": 8192, "d_model": 4096, "n_ffn": 256,
         "n_zero": 128, "d_ff": 1536, "top_k": 8, "scaling": 1.0, "skew": 2.0, "accumulate": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gmm", "gmm", "adamw", "layer"])
    if op == "gmm":
        f32 = rng.random() < 0.3
        while True:
            groups, rows = _log(rng, 1, 256), _log(rng, 1, 40960)
            n, k = _log(rng, 24, 6144), _log(rng, 24, 6144)
            if rng.random() < 0.7:
                n, k = max(8, n // 8 * 8), max(8, k // 8 * 8)
            if groups * n * k <= 1.6e9 and rows * n * k <= (4e10 if f32 else 2.5e11):
                break
        form = rng.choice(["fwd", "dx", "dw"])
        acc = rng.random() < 0.3
        return {"op": "gmm", "form": form, "dtype": "f32" if f32 else "bf16",
                "out": "f32" if f32 or rng.random() < 0.3 else "bf16", "groups": groups, "rows": rows,
                "spare": rng.choice([0, rng.randrange(1, 2000)]), "n": n, "k": k,
                "zipf": rng.choice([0.0, 0.7, 1.2]), "accumulate": acc}
    if op == "adamw":
        tensors = _log(rng, 1, 200)
        return {"op": "adamw", "bits": rng.choice([8, 32]), "tensors": tensors,
                "total": tensors + _log(rng, 500, 350_000_000),
                "dtype": (dt := rng.choice(["bf16", "f32"])), "grad": rng.choice([dt, "f32"]),
                "master": dt == "bf16" and rng.random() < 0.7, "decay": rng.choice([0.0, 0.01, 0.1])}
    f32 = rng.random() < 0.3
    while True:
        t, d, ff = _log(rng, 1, 8192), 64 * _log(rng, 1, 64), 64 * _log(rng, 1, 24)
        n_ffn, n_zero = _log(rng, 1, 256), rng.choice([0, _log(rng, 1, 128)])
        top_k = min(_log(rng, 1, 12), n_ffn + n_zero)
        if n_ffn * d * ff <= 1.6e9 and t * top_k * d * ff <= (2e10 if f32 else 2.7e11):
            break
    return {"op": "layer", "dtype": "f32" if f32 else "bf16", "tokens": t, "d_model": d, "n_ffn": n_ffn,
            "n_zero": n_zero, "d_ff": ff, "top_k": top_k, "scaling": rng.choice([1.0, 2.5]),
            "skew": rng.choice([0.0, 1.0, 2.0]), "accumulate": rng.random() < 0.25}


def _touched(groups, rows):
    """Experts that hold rows, on average, when `rows` fall on `groups` evenly."""
    return groups * (1.0 - (1.0 - 1.0 / groups) ** rows)


def work(case):
    c = case
    if c["op"] == "gmm":
        es, eo = SIZE[c["dtype"]], SIZE[c["out"]]
        rows, n, k = c["rows"], c["n"], c["k"]
        again = 2 if c["accumulate"] else 1     # the old value is read too
        if c["form"] == "dw":
            b = rows * (n + k) * es + c["groups"] * n * k * eo * again
        else:
            wide, narrow = (k, n) if c["form"] == "fwd" else (n, k)
            b = rows * wide * es + _touched(c["groups"], rows) * n * k * es + rows * narrow * eo * again
        return {"bytes": b, "flops": 2.0 * rows * n * k}
    if c["op"] == "adamw":
        each = 2 * SIZE[c["dtype"]] + SIZE[c["grad"]] + (16 if c["bits"] == 32 else 4 + 16 / Q_BLOCK)
        if c["master"]:
            each += 8 - SIZE[c["dtype"]]        # the rounded copy is only written
        return {"bytes": each * c["total"], "flops": 12.0 * c["total"]}
    es = SIZE[c["dtype"]]
    t, d, ff, e = c["tokens"], c["d_model"], c["d_ff"], c["n_ffn"] + c["n_zero"]
    rows = t * c["top_k"] * c["n_ffn"] / e
    weights, again = 3.0 * c["n_ffn"] * d * ff * es, 2 if c["accumulate"] else 1
    b = 3 * t * d * es + (1 + again) * (weights + e * d * es) + 2 * t * e * 4 + t * c["top_k"] * 20
    # three products to recompute gate, up and the gradient at H, two for the rows, three for the weights
    return {"bytes": b, "flops": 2.0 * rows * d * ff * 8 + 2 * 2.0 * t * e * d}


# ---- inputs


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _counts(c, seed):
    """How many rows each expert has: even or Zipf-distributed, in a random order."""
    g = _gen(seed, "cpu")
    q = torch.arange(1, c["groups"] + 1, dtype=torch.float64).pow(-c["zipf"])
    q = q[torch.randperm(c["groups"], generator=g)]
    at = torch.multinomial(q / q.sum(), c["rows"], replacement=True, generator=g)
    return torch.bincount(at, minlength=c["groups"])


def _prepare_gmm(c, seed):
    g = _gen(seed, "cuda")

    def normal(shape, std, dtype):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    dt, out = DTYPES[c["dtype"]], DTYPES[c["out"]]
    counts = _counts(c, seed)
    m, n, k = c["rows"] + c["spare"], c["n"], c["k"]
    offsets = torch.zeros(c["groups"] + 1, dtype=torch.int32)
    offsets[1:] = counts.cumsum(0)
    s = {"counts": counts.tolist(), "offsets": offsets.cuda()}
    if c["form"] == "fwd":
        s["lhs"], s["rhs"], shape = normal((m, k), 1.0, dt), normal((c["groups"], n, k), k ** -0.5, dt), (m, n)
    elif c["form"] == "dx":
        s["lhs"], s["rhs"], shape = normal((m, n), 1.0, dt), normal((c["groups"], n, k), n ** -0.5, dt), (m, k)
    else:
        s["lhs"], s["rhs"], shape = normal((m, n), 1.0, dt), normal((m, k), 1.0, dt), (c["groups"], n, k)
    s["out"] = normal(shape, 1.0, out) if c["accumulate"] else torch.zeros(shape, dtype=out, device="cuda")
    return s


def _lengths(c):
    """Tensor lengths that add up to the total, each a different odd share of it."""
    t = c["tensors"]
    share = [1.0 + (i * 7 % 5) for i in range(t)] if t > 3 else [1.0] * t
    whole = sum(share)
    got = [max(1, int(c["total"] * x / whole)) for x in share]
    got[-1] = max(1, got[-1] + c["total"] - sum(got))
    return got


def _to_blocks(x):
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % Q_BLOCK)).view(-1, Q_BLOCK)


def _prepare_adamw(c, seed):
    g = _gen(seed, "cuda")

    def normal(n, std):
        return torch.randn(n, generator=g, device="cuda").mul_(std)

    def tensor(i, n):
        w = normal(n, 0.02)
        t = {"param": w.to(DTYPES[c["dtype"]]), "grad": normal(n, 1e-3).to(DTYPES[c["grad"]]),
             "decay": c["decay"] if i % 2 == 0 else 0.0}
        if c["master"]:
            t["master"] = w
        m, r = normal(n, 3e-4), normal(n, 1e-3).abs_().add_(1e-5)
        if c["bits"] == 32:
            t["m"], t["v"] = m, r.square_()
        else:
            for name, x in (("m", m), ("v", r)):     # the second moment is kept as its root
                b = _to_blocks(x)
                scale = b.abs().amax(1) / Q_MAX
                t[name] = (b / scale[:, None]).to(F8).view(-1)[:n].clone()
                t[name + "_scale"] = scale
        return t

    return {"tensors": [tensor(i, n) for i, n in enumerate(_lengths(c))],
            "hyper": {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "seed": seed & 0x7FFFFFFF},
            "step": torch.tensor([100, 0, 0, 0], dtype=torch.int32, device="cuda"),
            "grad_scale": torch.tensor([0.7], device="cuda")}


def _prepare_layer(c, seed):
    g = _gen(seed, "cuda")
    dt = DTYPES[c["dtype"]]
    t, d, ff, n_ffn, e, k = c["tokens"], c["d_model"], c["d_ff"], c["n_ffn"], c["n_ffn"] + c["n_zero"], c["top_k"]

    def normal(shape, std, dtype=dt):
        return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)

    s = {"x": normal((t, d), 1.0), "dy": normal((t, d), 1.0), "w_router": normal((e, d), d ** -0.5),
         "w_gate": normal((n_ffn, ff, d), d ** -0.5), "w_up": normal((n_ffn, ff, d), d ** -0.5),
         "w_down": normal((n_ffn, d, ff), ff ** -0.5)}
    # what the forward pass leaves: logits, selection, gates, and the rows grouped by expert
    offset = normal((e,), c["skew"], F32)
    s["logits"] = s["x"].float() @ s["w_router"].float().t() + offset
    p = torch.softmax(s["logits"], 1)
    idx = torch.topk(p, k, dim=1).indices.sort(dim=1).values
    s["topk_idx"] = idx.to(torch.int32)
    s["topk_gate"] = c["scaling"] * p.gather(1, idx)
    flat = idx.reshape(-1)
    perm = torch.sort(flat, stable=True).indices
    s["perm"] = perm.to(torch.int32)
    s["inv_perm"] = torch.empty_like(perm).scatter_(0, perm, torch.arange(t * k, device="cuda")).to(torch.int32)
    counts = torch.bincount(flat, minlength=e)
    s["offsets"] = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    s["offsets"][1:] = counts.cumsum(0)
    s["counts"] = counts[:n_ffn].tolist()
    for name, like in (("dw_router", "w_router"), ("dw_gate", "w_gate"), ("dw_up", "w_up"), ("dw_down", "w_down")):
        s[name] = normal(s[like].shape, 1.0) if c["accumulate"] else torch.zeros_like(s[like])
    return s


def prepare(case, seed):
    make = {"gmm": _prepare_gmm, "adamw": _prepare_adamw, "layer": _prepare_layer}[case["op"]]
    return {"case": case, **make(case, seed)}


# ---- the plain forms


def _plain_gmm(s):
    """fwd: out[p] = lhs[p] W_e^T; dx: out[p] = lhs[p] W_e; dw: out[e] = sum over its rows of lhs[p]^T rhs[p]."""
    c, out, counts = s["case"], s["out"], s["counts"]
    rows = c["rows"]
    lhs = torch.split(s["lhs"][:rows], counts)
    if c["form"] == "dw":
        rhs = torch.split(s["rhs"][:rows], counts)
        new = [x.float().t() @ y.float() for x, y in zip(lhs, rhs)]
        [o.copy_(o.float() + v if c["accumulate"] else v) for o, v in zip(out, new)]
        return out
    new = torch.cat([x.float() @ (w.float().t() if c["form"] == "fwd" else w.float())
                     for x, w in zip(lhs, s["rhs"])])
    out[:rows] = (out[:rows].float() + new if c["accumulate"] else new).to(out.dtype)
    return out


def _mix(x):
    """A 32-bit integer hash (two rounds of xor-shift and multiply) on int64 tensors or ints."""
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & MASK32
    x = ((x ^ (x >> 15)) * 0x846CA68B) & MASK32
    return x ^ (x >> 16)


def _random16(seed, step, tensor, n):
    """Two numbers in [0, 1) for each element, multiples of 2^-16, from its place alone."""
    base = _mix((seed + 0x9E3779B9 * step) & MASK32)
    key = _mix((base + tensor) & MASK32)
    i = torch.arange(n, device="cuda")
    h = _mix((i + key + 0x9E3779B9 * (i >> 32)) & MASK32)
    return (h & 0xFFFF).float() / 65536, (h >> 16).float() / 65536


def _grid(y):
    """The e4m3 values next to y >= 0 (below or equal, above), for y up to 448."""
    e = torch.frexp(y).exponent - 1
    ulp = torch.ldexp(torch.ones_like(y), e.clamp(min=-6) - 3)
    low = torch.floor(y / ulp) * ulp
    return low, (low + ulp).clamp(max=Q_MAX)


def _quantise(x, u, square):
    """Codes and block scales of x, rounded up or down at random so that the mean of the code (of its
    square, for the root of the second moment) is the value."""
    n = x.numel()
    b = _to_blocks(x)
    top = b.abs().amax(1)
    scale = top / Q_MAX
    inv = torch.where(top > 2.0 ** -100, Q_MAX / top, torch.zeros_like(top))
    y = (b.abs() * inv[:, None]).clamp(max=Q_MAX).view(-1)[:n]
    low, high = _grid(y)
    if square:
        up = u * (high * high - low * low) < y * y - low * low
    else:
        up = u * (high - low) < y - low
    q = torch.where(up, high, low)
    if square:
        q = torch.where(y > 0, q.clamp(min=2.0 ** -9), q)
    return torch.copysign(q, x).to(F8), scale


def _held(q, scale):
    """The values that codes and scales stand for."""
    return (_to_blocks(q.float()) * scale[:, None]).view(-1)[:q.numel()]


def _plain_adamw(s):
    c, h = s["case"], s["hyper"]
    b1, b2 = h["beta1"], h["beta2"]
    step = s["step"][0] + 1
    t = step.double()
    c1, c2 = (1 - b1 ** t).float(), (1 - b2 ** t).float()

    def one(i, w):
        at = w.get("master", w["param"])
        p, g = at.float(), w["grad"].float() * s["grad_scale"]
        if c["bits"] == 32:
            m, v = w["m"], w["v"]
        else:
            m, v = _held(w["m"], w["m_scale"]), _held(w["v"], w["v_scale"]).square()
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g * g
        p = p * (1 - h["lr"] * w["decay"]) - h["lr"] * (m / c1) / (torch.sqrt(v / c2) + h["eps"])
        if c["bits"] == 32:
            w["m"].copy_(m), w["v"].copy_(v)
        else:
            um, uv = _random16(h["seed"], step.long(), i, p.numel())
            for name, new, u, square in (("m", m, um, False), ("v", torch.sqrt(v), uv, True)):
                q, scale = _quantise(new, u, square)
                w[name].copy_(q), w[name + "_scale"].copy_(scale)
        w["param"].copy_(p)
        if "master" in w:
            w["master"].copy_(p)

    [one(i, w) for i, w in enumerate(s["tensors"])]
    s["step"][0] += 1
    return _adamw_outputs(s)


def _adamw_outputs(s):
    """Everything that the step has written, in as few outputs as there are kinds of tensors."""
    if len(s["tensors"]) <= 8:
        kept = [{k: v for k, v in w.items() if k not in ("grad", "decay")} for w in s["tensors"]]
        return {"tensors": kept, "step": s["step"][:1]}
    names = [k for k in s["tensors"][0] if k not in ("grad", "decay")]

    def joined(k):
        if s["tensors"][0][k].dtype == F8:
            return torch.cat([w[k].view(torch.uint8) for w in s["tensors"]]).view(F8)
        return torch.cat([w[k] for w in s["tensors"]])

    return {**{k: joined(k) for k in names}, "step": s["step"][:1]}


def _plain_layer(s):
    c = s["case"]
    k, n_ffn, rows = c["top_k"], c["n_ffn"], sum(s["counts"])
    x, dy, idx = s["x"].float(), s["dy"].float(), s["topk_idx"].long()
    gate = s["topk_gate"]
    at = s["perm"][:rows].long()                       # assignments of the FFN experts, by expert
    xs, dys, gs = x[at // k], dy[at // k], gate.view(-1)[at]

    def expert(e, xe, dye, ge):
        wg, wu, wd = s["w_gate"][e].float(), s["w_up"][e].float(), s["w_down"][e].float()
        z, u, dh = xe @ wg.t(), xe @ wu.t(), dye @ wd
        sig = torch.sigmoid(z)
        h = z * sig * u
        dgate = (dh * h).sum(1)
        dh = dh * ge[:, None]
        dz, du = dh * u * sig * (1 + z * (1 - sig)), dh * z * sig
        for name, dw in (("dw_gate", dz.t() @ xe), ("dw_up", du.t() @ xe), ("dw_down", dye.t() @ (h * ge[:, None]))):
            s[name][e] = dw + s[name][e].float() if c["accumulate"] else dw
        return dz @ wg + du @ wu, dgate

    per = torch.split(xs, s["counts"]), torch.split(dys, s["counts"]), torch.split(gs, s["counts"])
    both = [expert(e, *parts) for e, parts in enumerate(zip(*per))]
    dx_rows, dgate_rows = torch.cat([b[0] for b in both]), torch.cat([b[1] for b in both])
    zero = idx >= n_ffn
    dgate = torch.where(zero, (x * dy).sum(1, keepdim=True), torch.zeros_like(gate)).view(-1)
    dgate[at] = dgate_rows
    dgate = dgate.view(-1, k)
    dx = dy * (gate * zero).sum(1, keepdim=True)
    dx.index_add_(0, at // k, dx_rows)
    p = torch.softmax(s["logits"], 1)
    dp = torch.zeros_like(p).scatter_(1, idx, c["scaling"] * dgate)
    dlogits = p * (dp - (p * dp).sum(1, keepdim=True))
    dx += dlogits @ s["w_router"].float()
    dwr = dlogits.t() @ x
    s["dw_router"].copy_(dwr + s["dw_router"].float() if c["accumulate"] else dwr)
    return {"dx": dx.to(s["x"].dtype), "dgate": dgate, "dlogits": dlogits,
            **{n: s[n] for n in ("dw_router", "dw_gate", "dw_up", "dw_down")}}


# ---- the framework's operators


def _own_gmm(s):
    from sparse_moe_layer_03_amd import train as T
    c = s["case"]
    if "shape" not in s:
        s["shape"] = T.make_gmm_shape(c["form"], c["dtype"], c["groups"], c["rows"] + c["spare"], c["n"], c["k"],
                                      out_dtype=c["out"], accumulate=c["accumulate"])
        s["ws"] = torch.empty(T.moe_grouped_matmul_workspace_bytes(s["shape"]), dtype=torch.uint8, device="cuda")
    T.moe_grouped_matmul(s["shape"], s["offsets"], s["lhs"], s["rhs"], s["out"], s["ws"])
    return s["out"]


def _own_adamw(s):
    from sparse_moe_layer_03_amd import train as T
    if "list" not in s:
        h = s["hyper"]
        s["list"] = T.AdamwTensors([{**{k: v for k, v in w.items() if k != "decay"}, "weight_decay": w["decay"]}
                                    for w in s["tensors"]])
        s["params"] = T.make_adamw_params(h["lr"], h["beta1"], h["beta2"], h["eps"], s["case"]["bits"], h["seed"])
    T.moe_adamw(s["params"], s["list"], s["step"], grad_scale=s["grad_scale"])
    return _adamw_outputs(s)


def _own_layer(s):
    from sparse_moe_layer_03_amd import binding as B
    from sparse_moe_layer_03_amd import train as T
    c = s["case"]
    if "io" not in s:
        s["shape"] = B.make_shape(c["tokens"], c["d_model"], c["n_ffn"], c["n_zero"], c["d_ff"], c["top_k"],
                                  c["dtype"], c["scaling"])
        s["dx"], s["dgate"] = torch.empty_like(s["x"]), torch.empty_like(s["topk_gate"])
        s["dlogits"] = torch.empty_like(s["logits"])
        names = ("x", "w_router", "logits", "topk_idx", "topk_gate", "offsets", "perm", "inv_perm", "w_gate", "w_up",
                 "w_down", "dy", "dx", "dgate", "dlogits", "dw_router", "dw_gate", "dw_up", "dw_down")
        s["io"] = T.BackwardIO(**{n: s[n] for n in names}, accumulate=c["accumulate"])
        s["ws"] = torch.empty(T.moe_layer_backward_workspace_bytes(s["shape"]), dtype=torch.uint8, device="cuda")
    T.moe_layer_backward(s["shape"], s["io"], s["ws"])
    return {n: s[n] for n in ("dx", "dgate", "dlogits", "dw_router", "dw_gate", "dw_up", "dw_down")}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"gmm": _own_gmm, "adamw": _own_adamw, "layer": _own_layer}[op](state)
    return {"gmm": _plain_gmm, "adamw": _plain_adamw, "layer": _plain_layer}[op](state)


# ---- the definitions in 64 bits


def _exact_gmm(c, s):
    bounds = s["offsets"].tolist()
    out = s["out"].double() if s["out"].numel() < 2e8 or c["out"] == "f32" else s["out"].float()
    for e in range(c["groups"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi and c["form"] != "dw":
            continue
        x = s["lhs"][lo:hi].double()
        if c["form"] == "dw":
            v, to = torch.matmul(x.transpose(0, 1), s["rhs"][lo:hi].double()), out[e]
        else:
            w = s["rhs"][e].double()
            v, to = torch.matmul(x, w.transpose(0, 1) if c["form"] == "fwd" else w), out[lo:hi]
        if c["accumulate"]:
            to += v
        else:
            to.copy_(v)
    return out


def _exact_adamw(c, s):
    h, step = s["hyper"], int(s["step"][0]) + 1
    out = {**s, "tensors": []}
    for i, w in enumerate(s["tensors"]):
        n = w["param"].numel()
        block = torch.arange(n, device="cuda") // Q_BLOCK if c["bits"] == 8 else None
        m, v = w["m"].double(), w["v"].double()
        if c["bits"] == 8:
            m, v = m * w["m_scale"].double()[block], (v * w["v_scale"].double()[block]) ** 2
        g = w["grad"].double() * float(s["grad_scale"])
        m += (1 - h["beta1"]) * (g - m)
        v += (1 - h["beta2"]) * (g * g - v)
        del g
        p = w["master"].double() if c["master"] else w["param"].double()
        p *= 1 - h["lr"] * w["decay"]
        p -= h["lr"] * m / (1 - h["beta1"] ** step) / ((v / (1 - h["beta2"] ** step)).sqrt() + h["eps"])
        new = {"param": p}
        if c["master"]:
            new["master"] = p
        if c["bits"] == 32:
            new["m"], new["v"] = m, v
        else:       # the codes hang on rounding next to a border: only the scales have values of their own
            new["m"] = new["v"] = None
            for name, x in (("m", m.abs()), ("v", v.sqrt())):
                new[name + "_scale"] = _to_blocks(x).amax(1) / Q_MAX
        # laid out as the run's dict is
        out["tensors"].append({k: new[k] for k in w if k in new})
    if len(s["tensors"]) <= 8:
        return {"tensors": out["tensors"], "step": s["step"][:1] + 1}
    names = list(out["tensors"][0])
    return {**{k: None if out["tensors"][0][k] is None else torch.cat([w[k] for w in out["tensors"]])
               for k in names}, "step": s["step"][:1] + 1}


def _exact_layer(c, s):
    """By differentiating the definition: y = sum of gate * FFN(x) over the selected FFN experts, plus the
    identity experts' gates times x; gate = scaling * softmax(logits) at the selected experts."""
    t, k, n_ffn = c["tokens"], c["top_k"], c["n_ffn"]
    x = s["x"].double().requires_grad_()
    gate = s["topk_gate"].double().requires_grad_()
    dy, idx = s["dy"].double(), s["topk_idx"].long()
    y0 = (gate * (idx >= n_ffn)).sum(1, keepdim=True) * x
    y0.backward(dy)
    small = s["w_gate"].numel() < 2e8
    dws = {n: (s[n].double() if small else s[n].float()) for n in ("dw_gate", "dw_up", "dw_down")}
    for e in range(n_ffn):
        tok, slot = (idx == e).nonzero(as_tuple=True)
        w = [s[n][e].double().requires_grad_() for n in ("w_gate", "w_up", "w_down")]
        xe = x[tok]
        y = gate[tok, slot][:, None] * ((torch.nn.functional.silu(xe @ w[0].t()) * (xe @ w[1].t())) @ w[2].t())
        y.backward(dy[tok])
        for n, v in zip(dws, w):
            dws[n][e] = dws[n][e] + v.grad if c["accumulate"] else v.grad
    logits = s["logits"].double().requires_grad_()
    (c["scaling"] * torch.softmax(logits, 1).gather(1, idx)).backward(gate.grad)
    dl = logits.grad
    dwr = torch.matmul(dl.transpose(0, 1), s["x"].double())
    if c["accumulate"]:
        dwr += s["dw_router"].double()
    return {"dx": x.grad + dl @ s["w_router"].double(), "dgate": gate.grad, "dlogits": dl, "dw_router": dwr, **dws}


def exact(case, seed):
    c = dict(case)
    flops = work(c)["flops"]
    if flops > 8e12:
        return None
    s = prepare(c, seed)
    return {"gmm": _exact_gmm, "adamw": _exact_adamw, "layer": _exact_layer}[c["op"]](c, s)
