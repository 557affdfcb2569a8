"""The 8-bit products and the experts' FFN in the tile shapes of batches and
prefill (groups of some 100 to 300 rows and weights that fill the chip), more
tiles than a workgroup plans at once, more rows than the codes' grid, and wrong
routing arrays between guard bytes."""

import pytest
import torch

from sparse_moe_layer_03_amd import block as K
from tests.block_util import DT, codes, say
from tests.test_gpu_i8 import Ffn, check, check_quant
from tests.test_gpu_train_guards import Guarded
from tests.train_util import offsets_of

pytestmark = pytest.mark.gpu


# rows a group: 64 x 256, 128 x 256, 256 x 256, 320 x 192 and 256 x 256 tiles
@pytest.mark.parametrize("counts", [[5, 0, 23, 1] * 16, [24, 70, 130, 1] * 8, [200, 90, 256, 257, 0, 130] * 3,
                                    [256, 300, 320, 321, 250, 257, 271, 288, 304, 289, 0, 350], [512, 700, 1, 400] * 3])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("Kn", [16, 144, 1040])
def test_products_of_groups_that_fill_the_chip(counts, out, Kn):
    check(counts, 4100, Kn, out, spare=7, seed=len(counts))


# T, d, f, n, k: rows a group 12, 64, 150, 275, 400; the gate's and up tiles and the
# down tiles fill the chip
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,n,k,skew", [(200, 4096, 2048, 64, 4, 0.3), (512, 4096, 2048, 16, 2, 0.2), (1200, 4096, 2048, 16, 2, 0.2),
                                            (2200, 4096, 2048, 16, 2, 0.1), (2200, 4096, 1984, 16, 2, 0.0), (3200, 4096, 2048, 16, 2, 0.5)])
def test_expert_ffn_of_batches(dtype, T, d, f, n, k, skew):
    say(f"[ffn_i8] {dtype} T={T} d={d} f={f} n={n} k={k}")
    c = Ffn(T, d, f, n, 0, k, dtype, skew=skew)
    c.run()
    c.check()


def test_expert_ffn_of_prefill_with_identity_experts():
    """Rows in use go by the FFN experts' share: 270 a group of the 405."""
    c = Ffn(2160, 4096, 2048, 16, 8, 3, "bf16")
    say(f"[ffn_i8] rows {sum(c.counts[:16])} in {c.counts[:16]}")
    c.run()
    c.check()


@pytest.mark.parametrize("counts,N", [([16500, 0, 16500], 33028), ([3, 0, 9, 1, 2, 4, 1, 5] * 128, 5124)])
def test_more_tiles_than_a_workgroup_plans_at_once(counts, N):
    """More than 64 tiles for each workgroup: 16,900 of 256 x 256 over 256 of them,
    18,000 of 64 x 256."""
    say(f"[matmul_i8] {len(counts)} groups N={N}")
    g, G, M, Kn = torch.Generator(device="cuda").manual_seed(1), len(counts), sum(counts), 16
    a, w = codes((M, Kn), g), codes((G, N, Kn), g)
    sa, sw = torch.rand(M, generator=g, device="cuda") + 0.1, torch.randn((G, N), generator=g, device="cuda")
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    s = K.make_i8_shape("bf16", G, M, N, Kn)
    assert K.moe_matmul_i8_workspace_bytes(s) == 0
    K.moe_matmul_i8(s, offsets_of(counts), a, sa, w, sw, out)
    torch.cuda.synchronize()
    lo = 0
    for e, n in enumerate(counts):
        for i in range(lo, lo + n, 4096):
            part = slice(i, min(i + 4096, lo + n))
            # (16 products of codes: whole numbers below 2^24)
            want = ((a[part].float() @ w[e].float().t()) * sa[part, None] * sw[e]).bfloat16()
            assert torch.equal(out[part], want), (e, i)
        lo += n


@pytest.mark.parametrize("T,d,f,n,k", [(65536, 64, 8320, 2, 1), (400, 64, 2240, 1024, 16)])
def test_an_ffn_of_more_tiles_than_a_workgroup_plans_at_once(T, d, f, n, k):
    """Gate and up: 16,640 tiles of 256 x 128 columns; 18,000 of 64 x 128."""
    say(f"[ffn_i8] T={T} f={f} n={n}")
    c = Ffn(T, d, f, n, 0, k, "bf16")
    c.run()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,Kn", [(40001, 40), (40001, 1000), (9001, 1500), (9001, 4000), (9001, 8192), (2300, 9000), (2300, 33000)])
def test_codes_of_more_rows_than_the_grid_holds(dtype, M, Kn):
    """Up to 8192 workgroups, of 4 rows each up to 1024 columns; 2048 of the long rows'."""
    g = torch.Generator(device="cuda").manual_seed(M)
    check_quant(torch.randn((M, Kn), generator=g, device="cuda").to(DT[dtype]))


# ---- wrong routing arrays


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,d,f,n,z,k", [(40, 128, 64, 6, 2, 3), (1200, 4096, 1024, 16, 4, 2)])
@pytest.mark.parametrize("wrong", ["perm", "offsets", "last"])
def test_wrong_routing_arrays_write_nothing_outside(dtype, T, d, f, n, z, k, wrong):
    """Permutations and offsets out of range, and descending ones: every array lies
    between guard bytes, and no byte outside the outputs changes."""
    say(f"[guards] ffn_i8 {dtype} T={T} wrong {wrong}")
    c = Ffn(T, d, f, n, z, k, dtype)
    g = torch.Generator(device="cuda").manual_seed(4)
    if wrong == "perm":
        c.perm[::5] = 1 << 30
        c.perm[1::7] = -3
        c.perm[2::11] = -(1 << 31)
    elif wrong == "offsets":
        c.offsets[1:-1] = torch.randint(-(1 << 31), (1 << 31) - 1, (n + z - 1,), generator=g, device="cuda").int()
        c.offsets[3], c.offsets[5] = 1 << 29, -5
    else:
        c.offsets[n] = (1 << 31) - 1
    kept = {name: Guarded(tuple(t.shape), t.dtype, fill=t) for name, t in
            (("x", c.x), ("perm", c.perm), ("offsets", c.offsets), *c.w.items())}
    y, ws = Guarded((T * k, d), c.dt), Guarded((c.ws.numel(),), torch.uint8)
    K.moe_expert_ffn_i8(c.s, K.FfnI8IO(y_perm=y.t, **{name: a.t for name, a in kept.items()}), ws.t)
    torch.cuda.synchronize()
    for name, a in kept.items():
        a.check(name, written=False)
    ws.check("ws"), y.check("y_perm")


@pytest.mark.parametrize("N,Kn", [(72, 160), (70, 161), (520, 6144), (4096, 128)])
@pytest.mark.parametrize("off", [[0, 1 << 30, -7, 200, 300], [-(1 << 31), (1 << 31) - 1, 0, 90, 1 << 29], [300, 200, 100, 50, 0],
                                 [0, 300, 0, 300, 0], [290, 290, 290, 310, 400]])
def test_wrong_offsets_of_products_write_nothing_outside(off, N, Kn):
    say(f"[guards] matmul_i8 N={N} K={Kn} offsets {off}")
    g, G, M = torch.Generator(device="cuda").manual_seed(2), len(off) - 1, 300
    s = K.make_i8_shape("bf16", G, M, N, Kn)
    a, w = (Guarded(n, torch.int8, fill=codes(n, g)) for n in ((M, Kn), (G, N, Kn)))
    sa, sw = (Guarded(n, torch.float32, fill=torch.rand(n, generator=g, device="cuda")) for n in ((M,), (G, N)))
    offsets = Guarded((G + 1,), torch.int32, fill=torch.tensor(off, dtype=torch.int32))
    out, ws = Guarded((M, N), torch.bfloat16), Guarded((K.moe_matmul_i8_workspace_bytes(s),), torch.uint8)
    K.moe_matmul_i8(s, offsets.t, a.t, sa.t, w.t, sw.t, out.t, ws.t)
    torch.cuda.synchronize()
    for name, v in (("a", a), ("sa", sa), ("w", w), ("sw", sw), ("offsets", offsets)):
        v.check(name, written=False)
    ws.check("ws"), out.check("out")
