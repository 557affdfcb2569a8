"""moe_adamw against the step in 64 bits: types, 32-bit copies, many tensors,
odd lengths, both kinds of moments, skipped steps, learning-rate scales,
streams and captured graphs; the 8-bit moments' codes bit by bit against the
same rounding in elementary operations, and the means they keep."""

import pytest
import torch

from sparse_moe_layer_03_amd import binding as B
from sparse_moe_layer_03_amd import train as T
from tests.train_util import U

pytestmark = pytest.mark.gpu
BF16, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-8)


def say(*a):
    print(*a, flush=True)


def blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % 256)).view(-1, 256)


def make(lengths, p_dt=BF16, g_dt=BF16, master=True, bits=32, seed=0, fresh=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(lengths):
        w = torch.randn(n, generator=g, device="cuda") * 0.1
        t = {"param": w.to(p_dt), "grad": (torch.randn(n, generator=g, device="cuda") * 1e-2).to(g_dt),
             "weight_decay": 0.1 * (i % 3)}
        if master:
            t["master"] = w
        m = torch.randn(n, generator=g, device="cuda") * 1e-3
        r = torch.rand(n, generator=g, device="cuda") * 1e-2
        if fresh:
            m, r = m * 0, r * 0
        if bits == 32:
            t["m"], t["v"] = m, r * r
        else:
            for name, x in (("m", m), ("v", r)):
                b = blocks(x)
                sc = b.abs().amax(1) / 448
                q = b / sc.clamp(min=1e-30)[:, None]
                t[name], t[name + "_scale"] = q.view(-1)[:n].to(F8).clone(), sc
        out.append(t)
    return out


def held(t, name):
    """A moment in 64 bits."""
    x = t[name].double()
    if t["m"].dtype == F32:
        return x
    x = x * t[name + "_scale"].double().repeat_interleave(256)[:x.numel()]
    return x * x if name == "v" else x


def reference(t, step, gs=1.0, lr_scale=1.0, h=HYPER):
    """p, m, v of the step in 64 bits, and the magnitude that the update's
    error is measured by: m = b1 m0 + (1 - b1) g may cancel, and its terms'
    roundings, each relative to the term, stay; lr / denominator times them
    is what reaches p.  So the bound has |b1 m0| + |(1 - b1) g| where the
    update has their sum."""
    b1, b2, lr = h["beta1"], h["beta2"], h["lr"] * lr_scale
    p = (t["master"] if "master" in t else t["param"]).double()
    g = t["grad"].double() * gs
    m = b1 * held(t, "m") + (1 - b1) * g
    v = b2 * held(t, "v") + (1 - b2) * g * g
    down = (1 - b1 ** step) * ((v / (1 - b2 ** step)).sqrt() + h["eps"])
    terms = b1 * held(t, "m").abs() + (1 - b1) * g.abs()
    return p * (1 - lr * t["weight_decay"]) - lr * m / down, m, v, lr * terms / down


def clone(ts):
    return [{k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in t.items()} for t in ts]


def step_state(n):
    s = T.new_adamw_state()
    s[0] = n
    return s


# A step takes fewer than 16 fp32 operations to each result, each off by at
# most a step of the largest value that enters the sum.
EPS = 16 * 2.0 ** -23


def check(before, after, step, gs=1.0, lr_scale=1.0, h=HYPER):
    for i, (b, a) in enumerate(zip(before, after)):
        p, m, v, up = reference(b, step, gs, lr_scale, h)
        g = b["grad"].double() * gs
        value = (a["master"] if "master" in a else a["param"]).double()
        tol = EPS * (p.abs() + up.abs() + value.abs())
        if "master" not in a:
            tol = tol + U[a["param"].dtype] * p.abs() * 1.01
        assert ((value - p).abs() <= tol).all(), i
        if "master" in a:
            assert torch.equal(a["param"], a["master"].to(a["param"].dtype)), i
        if a["m"].dtype == F32:
            assert ((a["m"].double() - m).abs() <= EPS * (m.abs() + g.abs() + held(b, "m").abs())).all(), i
            assert ((a["v"].double() - v).abs() <= EPS * v).all(), i
        assert torch.equal(a["grad"], b["grad"])


LENGTHS = [1, 7, 8, 9, 255, 256, 257, 2047, 2048, 2049, 10007]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dt,g_dt,master", [(F32, F32, False), (BF16, BF16, True), (BF16, F32, True),
                                              (BF16, BF16, False), (F32, BF16, False), (F32, F32, True)])
@pytest.mark.parametrize("step", [0, 1, 5000])
def test_step(bits, p_dt, g_dt, master, step):
    say(f"[adamw] bits={bits} {p_dt} {g_dt} master={master} step={step}")
    ts = make(LENGTHS, p_dt, g_dt, master, bits, seed=step)
    before, state = clone(ts), step_state(step)
    T.moe_adamw(T.make_adamw_params(**HYPER, state_bits=bits, seed=9), T.AdamwTensors(ts), state)
    torch.cuda.synchronize()
    assert state.tolist() == [step + 1, 0, 0, 0]
    check(before, ts, step + 1)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [47, 48, 49, 97, 200])
def test_many_tensors(bits, count):
    # over the border of one launch's list; empty tensors among them
    lengths = [(i * 37) % 700 if i % 11 else 0 for i in range(count)]
    ts = make(lengths, BF16, BF16, True, bits, seed=count)
    ts = [t if t["param"].numel() else {**t, "weight_decay": 0.0} for t in ts]
    before, state = clone(ts), T.new_adamw_state()
    T.moe_adamw(T.make_adamw_params(**HYPER, state_bits=bits), T.AdamwTensors(ts), state)
    torch.cuda.synchronize()
    assert state.tolist() == [1, 0, 0, 0]
    check(before, ts, 1)


def test_more_chunks_than_workgroups():
    ts = make([9_000_001, 300, 2_500_000], BF16, BF16, True, 32)
    before, state = clone(ts), T.new_adamw_state()
    T.moe_adamw(T.make_adamw_params(**HYPER), T.AdamwTensors(ts), state)
    torch.cuda.synchronize()
    check(before, ts, 1)


@pytest.mark.parametrize("bits", [32, 8])
def test_only_empty_tensors_still_count_a_step(bits):
    ts = make([0, 0], BF16, BF16, True, bits)
    state = T.new_adamw_state()
    T.moe_adamw(T.make_adamw_params(**HYPER, state_bits=bits), T.AdamwTensors(ts), state)
    assert state.tolist() == [1, 0, 0, 0]


@pytest.mark.parametrize("bits", [32, 8])
def test_scales_and_skipped_steps(bits):
    ts = make([5000, 33], bits=bits)
    tensors, params = T.AdamwTensors(ts), T.make_adamw_params(**HYPER, state_bits=bits)
    state = T.new_adamw_state()
    before = clone(ts)
    for bad in (float("nan"), float("inf"), -float("inf")):
        T.moe_adamw(params, tensors, state, grad_scale=torch.tensor([bad], device="cuda"))
    torch.cuda.synchronize()
    assert state.tolist() == [0, 3, 0, 0]
    for b, a in zip(before, ts):
        for k in b:
            if isinstance(b[k], torch.Tensor):
                assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    gs, ls = torch.tensor([0.3], device="cuda"), torch.tensor([0.5], device="cuda")
    T.moe_adamw(params, tensors, state, grad_scale=gs, lr_scale=ls)
    torch.cuda.synchronize()
    assert state.tolist() == [1, 3, 0, 0]
    check(before, ts, 1, gs=float(gs), lr_scale=0.5)


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_replays_count_their_steps(bits):
    ts = make([70_001, 5], bits=bits)
    twin = clone(ts)
    params, state, twin_state = T.make_adamw_params(**HYPER, state_bits=bits, seed=3), T.new_adamw_state(), \
        T.new_adamw_state()
    tensors, twins = T.AdamwTensors(ts), T.AdamwTensors(twin)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.moe_adamw(params, tensors, state)
    for k in range(4):
        graph.replay()
        T.moe_adamw(params, twins, twin_state)
        torch.cuda.synchronize()
        assert state.tolist() == twin_state.tolist() == [k + 1, 0, 0, 0]
        for a, b in zip(ts, twin):
            for n in a:
                if isinstance(a[n], torch.Tensor):
                    assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), (k, n)


def mix(x):
    x = ((x ^ (x >> 16)) * 0x7FEB352D) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x846CA68B) & 0xFFFFFFFF
    return x ^ (x >> 16)


def test_8_bit_codes_follow_their_rounding():
    # every code is a neighbour of its value, the one that the random number
    # picks wherever the fp32 result cannot change the choice
    n, step, seed, place = 20_011, 77, 5, 2
    ts = make([3, 600, n], BF16, F32, True, 8)
    before = clone(ts)
    T.moe_adamw(T.make_adamw_params(**HYPER, state_bits=8, seed=seed), T.AdamwTensors(ts), step_state(step - 1))
    torch.cuda.synchronize()
    _, m, v, _ = reference(before[place], step)
    key = mix((mix((seed + 0x9E3779B9 * step) & 0xFFFFFFFF) + place) & 0xFFFFFFFF)
    h = mix((torch.arange(n, device="cuda") + key) & 0xFFFFFFFF)
    grid = torch.arange(127, device="cuda", dtype=torch.uint8).view(F8).double()
    for name, x, u in (("m", m, (h & 0xFFFF).double() / 65536), ("v", v.sqrt(), (h >> 16).double() / 65536)):
        top = blocks(x.abs()).amax(1)
        scale = ts[place][name + "_scale"].double()
        assert ((scale - top / 448).abs() <= EPS * top).all()
        y = x.abs() / scale.repeat_interleave(256)[:n]
        low = (torch.searchsorted(grid, y, right=True) - 1).clamp(max=125)
        a, b = grid[low], grid[low + 1]
        q = ts[place][name].double()
        assert ((q == 0) | (torch.sign(q) == torch.sign(x))).all()
        q = q.abs()
        if name == "v":
            pick = torch.where(u * (b * b - a * a) < y * y - a * a, b, a)
            pick = torch.where(y > 0, pick.clamp(min=2.0 ** -9), pick)
            room = 64 * 2.0 ** -23 * (y * y + 1) / (b * b - a * a)
            near = (u - (y * y - a * a) / (b * b - a * a)).abs() <= room
        else:
            pick = torch.where(u * (b - a) < y - a, b, a)
            room = 64 * 2.0 ** -23 * (y + 1) / (b - a)
            near = (u - (y - a) / (b - a)).abs() <= room
        near |= (y - a <= EPS * (y + 1)) | (b - y <= EPS * (y + 1))
        assert near.float().mean() < 0.02
        assert (near | (q == pick)).all()
        assert ((q - y).abs() <= (b - a) * (1 + 1e-5)).all()


def test_8_bit_moments_keep_their_means():
    # gradients of one size: both moments must move towards them although one
    # step is far below half a code.  The mean over n elements is off by about
    # the codes' spacing (an eighth, a quarter for the square) / sqrt(n) a
    # step; 60 steps add up like sqrt(60), 6 standard deviations are allowed.
    n, steps = 1 << 16, 60
    ts = make([n], BF16, F32, True, 8, fresh=True)
    t = ts[0]
    t["m"].copy_(torch.full((n,), 100.0, device="cuda").to(F8)), t["v"].copy_(t["m"])
    t["m_scale"].fill_(1e-4), t["v_scale"].fill_(1e-4)
    t["grad"].fill_(1.4e-2)
    held_m, held_v = held(t, "m").mean().item(), held(t, "v").mean().item()
    h = dict(HYPER, beta1=0.99, beta2=0.995)
    state, params, tensors = T.new_adamw_state(), T.make_adamw_params(**h, state_bits=8), T.AdamwTensors(ts)
    for _ in range(steps):
        T.moe_adamw(params, tensors, state)
    want_m = 1.4e-2 + (held_m - 1.4e-2) * 0.99 ** steps
    want_v = 1.96e-4 + (held_v - 1.96e-4) * 0.995 ** steps
    room = 6 * (steps / n) ** 0.5
    assert abs(held(t, "m").mean().item() - want_m) <= room * 0.125 * want_m
    assert abs(held(t, "v").mean().item() - want_v) <= room * 0.25 * want_v


def test_8_bit_zero_blocks_and_small_values():
    # a block of zeros stays zero; a second moment above 0 stays above 0
    ts = make([1024], F32, F32, False, 8, fresh=True)
    t = ts[0]
    t["grad"].zero_()
    t["grad"][256], t["grad"][257] = 1.0, 1e-7
    T.moe_adamw(T.make_adamw_params(**HYPER, state_bits=8), T.AdamwTensors(ts), T.new_adamw_state())
    torch.cuda.synchronize()
    assert (t["m"][:256].float() == 0).all() and t["m_scale"][0] == 0 and t["v_scale"][0] == 0
    assert t["v"][256].float() == 448 and t["v"][257].float() == 2.0 ** -9
    assert torch.isfinite(t["param"]).all()


def test_non_finite_gradients_poison_their_block_alone():
    ts = make([1024], BF16, BF16, True, 8)
    before = clone(ts)
    t = ts[0]
    t["grad"][300] = float("nan")
    before[0]["grad"][300] = float("nan")
    T.moe_adamw(T.make_adamw_params(**HYPER, state_bits=8), T.AdamwTensors(ts), T.new_adamw_state())
    torch.cuda.synchronize()
    assert t["param"].isnan().nonzero().view(-1).tolist() == [300]
    assert t["m_scale"].isnan().nonzero().view(-1).tolist() == [1]
    assert t["v_scale"].isnan().nonzero().view(-1).tolist() == [1]


def test_another_stream():
    ts = make([5000], bits=32)
    before, state = clone(ts), T.new_adamw_state()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    T.moe_adamw(T.make_adamw_params(**HYPER), T.AdamwTensors(ts), state, stream=side)
    side.synchronize()
    check(before, ts, 1)


def test_refusals():
    ts = make([64])
    with pytest.raises(ValueError, match="grad"):
        T.AdamwTensors([{**ts[0], "grad": ts[0]["grad"][:10]}])
    with pytest.raises(ValueError, match=r"tensors\[0\].v"):
        T.AdamwTensors([{**ts[0], "v": ts[0]["v"].cpu()}])
    with pytest.raises(ValueError, match="contiguous"):
        T.AdamwTensors([{**ts[0], "m": torch.zeros(128, device="cuda")[::2]}])
    with pytest.raises(ValueError, match="m_scale"):
        T.AdamwTensors([{**ts[0], "m": ts[0]["m"].to(F8), "v": ts[0]["v"].to(F8)}])
    with pytest.raises(ValueError, match="state_bits"):
        T.moe_adamw(T.make_adamw_params(**HYPER, state_bits=8), T.AdamwTensors(ts), T.new_adamw_state())
    with pytest.raises(ValueError, match="state"):
        T.moe_adamw(T.make_adamw_params(**HYPER), T.AdamwTensors(ts), torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(B.MoeError, match="EINVAL"):
        T.moe_adamw(T.make_adamw_params(-1.0), T.AdamwTensors(ts), T.new_adamw_state())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("g", [1e-17, 1e-19, 3e-20])
def test_second_moment_below_the_normal_numbers(bits, g):
    # With beta1 = beta2 = 0 and p = 0 the step is lr g / (|g| + eps), here lr.
    # g^2 is a multiple of 2^-149, so rounded by at most 2^-150; half of that,
    # relative to g^2, is in its root.  The rest as in check().
    say(f"[adamw] bits={bits} gradient {g}")
    h = dict(lr=1e-2, beta1=0.0, beta2=0.0, eps=1e-30)
    ts = make([300], F32, F32, False, bits, fresh=True)
    ts[0]["param"].zero_()
    ts[0]["grad"].fill_(g)
    T.moe_adamw(T.make_adamw_params(**h, state_bits=bits), T.AdamwTensors(ts), T.new_adamw_state())
    torch.cuda.synchronize()
    off = (ts[0]["param"].double() / -h["lr"] - 1).abs().max().item()
    assert off <= EPS + 2.0 ** -150 / g ** 2 / 2, off


def test_refuses_arrays_that_overlap():
    ts = make([512, 512])
    T.AdamwTensors([ts[0], {**ts[1], "grad": ts[0]["grad"]}])               # read only: allowed
    T.AdamwTensors([ts[0], {**ts[1], "grad": ts[0]["grad"][:512]}])
    both = torch.zeros(1024, device="cuda")
    T.AdamwTensors([{**ts[0], "m": both[:512], "v": both[512:]}])           # side by side: allowed
    for bad in ([ts[0], ts[0]],                                             # a tied weight
                [ts[0], {**ts[1], "m": ts[0]["m"]}],
                [{**ts[0], "v": ts[0]["m"]}],
                [{**ts[0], "grad": ts[0]["master"]}],
                [ts[0], {**ts[1], "grad": ts[0]["v"]}],
                [{**ts[0], "m": both[:512], "v": both[511:1023]}],
                [{**ts[0], "m": both[256:768]}, {**ts[1], "grad": both[:512]}]):
        with pytest.raises(ValueError, match="overlap"):
            T.AdamwTensors(bad)
