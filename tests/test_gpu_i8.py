"""moe_quantize_rows, moe_matmul_i8 and moe_expert_ffn_i8 against the definition:
codes, scales and products bit by bit, the FFN within what a code next to a
border may change."""

import math

import pytest
import torch

from sparse_moe_layer_03_amd import binding as B
from sparse_moe_layer_03_amd import block as K
from tests.block_util import DT, U, codes, matmul_ref, quantise_ref, say
from tests.train_util import offsets_of

pytestmark = pytest.mark.gpu


def quantize(x, ldq=None):
    M, Kn = x.shape
    ldx = x.stride(0) if M > 1 else Kn
    s = K.make_quant_shape(x.dtype, M, Kn, ldx, ldq)
    q = torch.full((M, s.ldq), 99, dtype=torch.int8, device="cuda")[:, :Kn]
    scale = torch.full((M,), -1.0, device="cuda")
    K.moe_quantize_rows(s, x, q, scale)
    torch.cuda.synchronize()
    return q, scale


def check_quant(x, ldq=None):
    say(f"[quantize] {tuple(x.shape)} {x.dtype}")
    q, scale = quantize(x, ldq)
    wq, ws = quantise_ref(x)
    assert torch.equal(scale.isnan(), ws.isnan())
    assert torch.equal(scale[~scale.isnan()], ws[~ws.isnan()])
    assert torch.equal(q.double(), wq)
    return q, scale


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,Kn", [(1, 1), (3, 7), (5, 8), (257, 9), (64, 64), (33, 511), (7, 513), (100, 1001), (40, 2049),
                                  (9, 6144), (4, 8191), (3, 8200), (2, 32768), (2, 32771), (2, 131071), (5000, 24)])
def test_codes_and_scales(dtype, M, Kn):
    g = torch.Generator(device="cuda").manual_seed(M + Kn)
    check_quant(torch.randn((M, Kn), generator=g, device="cuda").to(DT[dtype]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quotients_on_and_next_to_borders(dtype):
    """Rows whose scale is a power of two, so that k + 1/2 is met exactly; and in
    fp32 values one step to either side."""
    half = torch.arange(-127, 127, device="cuda").float() + 0.5
    rows = []
    for e in (0, 5, -9, 60, -100):
        r = torch.cat([half, torch.tensor([127.0, -127.0, 0.0, -0.0], device="cuda")]) * 2.0 ** e
        rows.append(r)
        if dtype == "f32":
            for up in (math.inf, -math.inf):
                n = torch.nextafter(half, torch.full_like(half, up))
                rows.append(torch.cat([n, r[-4:] * 2.0 ** -e]) * 2.0 ** e)
    q, _ = check_quant(torch.stack(rows).to(DT[dtype]))
    assert (q[0, :254].double() == torch.round(half.double())).all()        # ties to even
    g = torch.Generator(device="cuda").manual_seed(1)
    tops = torch.rand((200, 1), generator=g, device="cuda") + 1
    k = torch.randint(-126, 126, (200, 300), generator=g, device="cuda") + 0.5
    x = (tops / 127 * k).to(DT[dtype])                                     # quotients next to borders
    x[:, :1] = tops.to(DT[dtype])
    check_quant(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_zeros_tiny_huge_and_non_finite_rows(dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((12, 100), generator=g, device="cuda")
    x[0] = 0
    x[1] = 0
    x[1, 50] = 1e-38
    x[2] *= 1e-40
    x[3] *= 1e38 / x[3].abs().max()
    x[4, 5] = math.inf
    x[5, 99] = math.nan
    x[6, 0] = -math.inf
    x[7] = torch.finfo(torch.bfloat16).max
    x[8] *= 1e-36
    q, scale = check_quant(x.to(DT[dtype]))
    assert scale[4].isnan() and scale[5].isnan() and scale[6].isnan() and (q[4:7] == 0).all()
    assert scale[0] == 2.0 ** -126 and (q[0] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_row_strides(dtype):
    g = torch.Generator(device="cuda").manual_seed(4)
    wide = torch.randn((50, 333), generator=g, device="cuda").to(DT[dtype])
    check_quant(wide[:, :301], 305)
    check_quant(wide[:, :8], 11)
    check_quant(wide[:, :3], 3)


# ---- products


def check(counts, N, Kn, out="bf16", spare=0, lda=None, ldc=None, seed=0, low=-127, offsets=True):
    say(f"[matmul_i8] groups={len(counts)} rows={sum(counts)} N={N} K={Kn} {out} lda={lda} ldc={ldc}")
    g = torch.Generator(device="cuda").manual_seed(seed)
    G, M = len(counts), sum(counts) + spare
    s = K.make_i8_shape(out, G, M, N, Kn, lda, ldc)
    a = codes((M, s.lda), g, low)[:, :Kn]
    w = codes((G, N, Kn), g, low)
    sa = torch.rand(M, generator=g, device="cuda") + 0.1
    sw = torch.randn((G, N), generator=g, device="cuda")
    c = torch.randn((M, s.ldc), generator=g, device="cuda").to(DT[out])[:, :N]
    old = c.clone()
    ws = torch.empty(K.moe_matmul_i8_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    K.moe_matmul_i8(s, offsets_of(counts) if offsets else None, a, sa, w, sw, c, ws)
    torch.cuda.synchronize()
    rows = sum(counts)
    want = matmul_ref(counts, a, sa, w, sw, DT[out])
    assert torch.equal(c[:rows], want), float((c[:rows].double() - want.double()).abs().max())
    assert torch.equal(c[rows:], old[rows:])


RAGGED = [0, 1, 63, 64, 65, 0, 257, 5, 128, 0]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N,Kn", [(64, 128), (96, 80), (1, 1), (37, 53), (8, 16), (264, 208), (130, 514), (4, 15), (128, 1040)])
def test_sizes(out, N, Kn):
    check(RAGGED, N, Kn, out, spare=3)


@pytest.mark.parametrize("counts", [[1], [0], [0, 0, 0], [1] * 40, [300], [0] * 7 + [33], [33] + [0] * 7, [700, 3, 300]])
@pytest.mark.parametrize("Kn", [192, 195])
def test_counts(counts, Kn):
    check(counts, 136, Kn, spare=2)


@pytest.mark.parametrize("counts,N,Kn", [([256] * 8 + [300, 0, 511, 17], 4096, 512), ([200] * 30, 2048, 256), ([1000], 8192, 1024),
                                         ([90] * 20, 1024, 384), ([2, 0, 3] * 50, 512, 2048)])
def test_every_tile_shape(counts, N, Kn):
    check(counts, N, Kn)
    check(counts, N, Kn - 1, "f32", spare=5)


@pytest.mark.parametrize("M", [1, 2, 16, 17, 63])
@pytest.mark.parametrize("N,Kn", [(512, 6144), (1000, 5121), (64, 131056), (3, 131071)])
def test_single_tokens_split_the_reduction(M, N, Kn):
    check([M], N, Kn, offsets=False)
    check([M, 0, 1], N, Kn, "f32", spare=1)


@pytest.mark.parametrize("N,Kn,lda,ldc", [(64, 128, 144, 72), (64, 128, 129, 64), (65, 128, 160, 67), (63, 100, 101, 77)])
def test_row_strides_of_products(N, Kn, lda, ldc):
    check(RAGGED, N, Kn, lda=lda, ldc=ldc, spare=2)
    check(RAGGED, N, Kn, "f32", lda=lda, ldc=ldc)


def test_largest_sums():
    """All codes -128 (which no quantised row holds) over the longest reduction."""
    Kn = 131071
    for k in (Kn, Kn // 16 * 16):
        a = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
        w = torch.full((1, 70, k), -128, dtype=torch.int8, device="cuda")
        s = K.make_i8_shape("f32", 1, 3, 70, k)
        out = torch.empty((3, 70), device="cuda")
        ws = torch.empty(K.moe_matmul_i8_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        one = torch.ones(70, device="cuda")
        K.moe_matmul_i8(s, None, a, one, w, one, out, ws)
        torch.cuda.synchronize()
        assert (out.double() == float(torch.tensor(16384.0 * k))).all()


def test_scales_of_nan_and_zero_reach_their_rows():
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((40, 96), generator=g, device="cuda").bfloat16()
    x[3, 7] = math.inf
    x[9] = 0
    q, sa = quantize(x)
    w, sw = codes((1, 64, 96), g), torch.ones((1, 64), device="cuda")
    out = torch.empty((40, 64), dtype=torch.bfloat16, device="cuda")
    K.moe_matmul_i8(K.make_i8_shape("bf16", 1, 40, 64, 96), None, q, sa, w, sw, out)
    torch.cuda.synchronize()
    assert out[3].isnan().all() and (out[9] == 0).all()
    assert torch.isfinite(out[[i for i in range(40) if i != 3]]).all()


def test_weights_behind_32_bits():
    G, N, Kn = 3, 2 ** 14, 2 ** 16 + 64 * 1024     # groups of 2^31 bytes
    w = torch.zeros((G, N, Kn - 1024), dtype=torch.int8, device="cuda")
    k = w.shape[2]
    w[2, N - 1, k - 1] = 3
    w[1, 5, 7] = 2
    a = torch.ones((3, k), dtype=torch.int8, device="cuda")
    one = torch.ones(G * N, device="cuda")
    out = torch.empty((3, N), device="cuda")
    s = K.make_i8_shape("f32", G, 3, N, k)
    ws = torch.empty(K.moe_matmul_i8_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    K.moe_matmul_i8(s, offsets_of([1, 1, 1]), a, one, w, one, out, ws)
    torch.cuda.synchronize()
    want = torch.zeros((3, N), device="cuda")
    want[2, N - 1], want[1, 5] = 3, 2
    assert torch.equal(out, want)


# ---- the experts' FFN


class Ffn:
    def __init__(self, T, d, f, n, z, k, dtype, seed=0, skew=0.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.s, self.dt = B.make_shape(T, d, n, z, f, k, dtype), DT[dtype]
        E = n + z
        self.x = torch.randn((T, d), generator=g, device="cuda").to(self.dt)
        score = torch.randn((T, E), generator=g, device="cuda") + skew * torch.randn(E, generator=g, device="cuda")
        flat = torch.topk(score, k, 1).indices.sort(1).values.reshape(-1)
        self.perm = torch.sort(flat, stable=True).indices.int()
        self.counts = torch.bincount(flat, minlength=E).tolist()
        self.offsets = offsets_of(self.counts)
        self.w = {}
        for name, a, b in (("gate", f, d), ("up", f, d), ("down", d, f)):
            self.w["w_" + name] = codes((n, a, b), g)
            self.w["s_" + name] = (torch.rand((n, a), generator=g, device="cuda") + 0.5) * (b ** -0.5 / 73)
        self.y = torch.full((T * k, d), 7.0, dtype=self.dt, device="cuda")
        self.ws = torch.empty(K.moe_expert_ffn_i8_workspace_bytes(self.s), dtype=torch.uint8, device="cuda")

    def io(self, **kw):
        return K.FfnI8IO(**{"x": self.x, "perm": self.perm, "offsets": self.offsets, "y_perm": self.y, **self.w, **kw})

    def run(self, **kw):
        K.moe_expert_ffn_i8(self.s, self.io(**kw), self.ws)
        torch.cuda.synchronize()
        return self.y

    def check(self):
        """H's products are exact up to their fp32 scaling; H may round the other
        way where it lies within silu's error (2^-19 of it, generous) of a border of
        its type.  Such an H moves its code by one step at most, or, being the row's
        largest, all codes of the row."""
        s, k, lo = self.s, self.s.top_k, 0
        q, sx = quantise_ref(self.x)
        f32 = self.dt == torch.float32
        for e in range(s.n_ffn):
            n = self.counts[e]
            if n == 0:
                continue
            tok = self.perm[lo:lo + n].long() // k
            z, u = ((q[tok] @ self.w["w_" + m][e].double().t()) * sx[tok, None].double() * self.w["s_" + m][e].double()
                    for m in ("gate", "up"))
            h = z / (1 + torch.exp(-z)) * u
            held = h.to(self.dt)
            eps = 2.0 ** -50 if f32 else 2.0 ** -19
            tiny = 1e-30
            loose = (h * (1 + eps) + tiny).to(self.dt) != (h * (1 - eps) - tiny).to(self.dt)
            hq, sh = quantise_ref(held)
            top = held.abs().amax(1, keepdim=True)
            whole = (loose & (held.abs() >= top * (1 - 2.0 ** -6))).any(1, keepdim=True)
            moved = (loose | whole).double()
            sd = self.w["s_down"][e].double()
            wd = self.w["w_down"][e].double()
            ref = (hq @ wd.t()) * sh[:, None].double() * sd
            bound = (moved @ wd.abs().t()) * sh[:, None].double() * sd * 1.02
            # a row whose scale moved: by a step of the type at most
            bound = bound + whole * 2 * U[self.dt] * ref.abs()
            err = (self.y[lo:lo + n].double() - ref).abs()
            assert (err <= bound + (U[self.dt] + 2.0 ** -21) * ref.abs() * 1.01 + 1e-30).all(), (e, float(err.max()))
            lo += n
        assert (self.y[lo:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,n,z,k,skew", [(1, 64, 64, 4, 0, 1, 0), (1, 192, 128, 8, 4, 3, 0), (37, 128, 192, 5, 3, 2, 1.0),
                                              (300, 256, 320, 16, 8, 4, 0), (130, 1024, 512, 64, 32, 8, 2.0), (2000, 256, 128, 4, 0, 2, 0),
                                              (16, 64, 64, 1, 0, 1, 0), (50, 64, 64, 300, 100, 12, 1.0)])
def test_expert_ffn(dtype, T, d, f, n, z, k, skew):
    say(f"[ffn_i8] {dtype} T={T} d={d} f={f} n={n} z={z} k={k}")
    c = Ffn(T, d, f, n, z, k, dtype, skew=skew)
    c.run()
    c.check()


def test_expert_ffn_takes_quantised_tokens():
    c = Ffn(70, 256, 192, 8, 4, 3, "bf16")
    want = c.run().clone()
    xq, xs = K.quantize_rows(c.x)
    c.y.fill_(7.0)
    assert torch.equal(c.run(x=None, xq=xq, x_scale=xs), want)


def test_expert_ffn_equals_its_parts():
    """The call against moe_quantize_rows and moe_matmul_i8, one expert."""
    c = Ffn(200, 256, 128, 1, 0, 1, "f32")
    y = c.run().clone()
    xq, xs = K.quantize_rows(c.x)
    z, u = (torch.empty((200, 128), device="cuda") for _ in range(2))
    s = K.make_i8_shape("f32", 1, 200, 128, 256)
    K.moe_matmul_i8(s, None, xq, xs, c.w["w_gate"], c.w["s_gate"], z)
    K.moe_matmul_i8(s, None, xq, xs, c.w["w_up"], c.w["s_up"], u)
    h = (z.double() / (1 + torch.exp(-z.double())) * u.double()).float()
    hq, hs = K.quantize_rows(h)
    out = torch.empty((200, 256), device="cuda")
    K.moe_matmul_i8(K.make_i8_shape("f32", 1, 200, 256, 128), None, hq, hs, c.w["w_down"], c.w["s_down"], out)
    torch.cuda.synchronize()
    assert (out - y).norm() <= 2e-3 * y.norm()      # (z and u are rounded to fp32 on the way)


def test_wrong_routing_arrays_stay_inside():
    """Permutations and offsets out of range give wrong rows, not accesses outside:
    the arrays lie in front of and behind others that must not change."""
    c = Ffn(40, 128, 64, 6, 2, 3, "bf16")
    keep = {n: t.clone() for n, t in c.w.items()}
    perm = c.perm.clone()
    perm[::5] = 1 << 30
    perm[1::7] = -3
    c.run(perm=perm)
    off = c.offsets.clone()
    off[3], off[5] = 1 << 29, -5
    c.run(offsets=off)
    assert all(torch.equal(c.w[n], keep[n]) for n in keep)


def test_streams_and_graphs():
    c = Ffn(130, 256, 192, 16, 8, 4, "bf16")
    want = c.run().clone()
    other = Ffn(130, 256, 192, 16, 8, 4, "bf16", seed=9)
    c.y.fill_(7.0)
    side = torch.cuda.Stream()
    K.moe_expert_ffn_i8(c.s, c.io(), c.ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(c.y, want)
    io = c.io()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.moe_expert_ffn_i8(c.s, io, c.ws)
    x0, p0, o0 = c.x.clone(), c.perm.clone(), c.offsets.clone()
    for x, p, o in ((other.x, other.perm, other.offsets), (x0, p0, o0), (other.x, other.perm, other.offsets)):
        c.x.copy_(x), c.perm.copy_(p), c.offsets.copy_(o)
        c.y.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        got = c.y.clone()
        c.y.fill_(7.0)
        K.moe_expert_ffn_i8(c.s, io, c.ws)
        torch.cuda.synchronize()
        assert torch.equal(got, c.y)
    c.x.copy_(x0), c.perm.copy_(p0), c.offsets.copy_(o0)
    c.y.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.y, want)
