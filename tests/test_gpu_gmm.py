"""moe_grouped_matmul against the products in 64 bits: the three forms, both
types, ragged and empty groups, odd sizes, row strides, accumulation, rows
behind the last group, split reductions, other streams, captured graphs."""

import pytest
import torch

from sparse_moe_layer_03_amd import binding as B
from sparse_moe_layer_03_amd import train as T
from tests.train_util import gmm_ref, offsets_of, sum_bound

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(*a):
    print(*a, flush=True)


def make(form, dtype, counts, N, K, spare=0, lda=None, ldc=None, out=None, accumulate=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    G, M = len(counts), sum(counts) + spare
    dt, od = DT[dtype], DT[out or dtype]
    s = T.make_gmm_shape(form, dtype, G, M, N, K, out_dtype=out or dtype, accumulate=accumulate,
                         lda=lda, ldc=ldc)

    def rows(width, ld, d):
        return torch.randn((M, ld), generator=g, device="cuda").to(d)[:, :width]

    def weights(d):
        return torch.randn((G, N, K), generator=g, device="cuda").to(d)

    a = lambda d: rows(K, s.lda, d)  # noqa: E731
    c = lambda d: rows(N, s.ldc, d)  # noqa: E731
    if form == "fwd":
        return s, a(dt), weights(dt), c(od)
    if form == "dx":
        return s, c(dt), weights(dt), a(od)
    return s, c(dt), a(dt), weights(od)


def run(s, counts, lhs, rhs, out, stream=None):
    ws = torch.empty(T.moe_grouped_matmul_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    T.moe_grouped_matmul(s, offsets_of(counts), lhs, rhs, out, ws, stream=stream)
    torch.cuda.synchronize()


def check(form, dtype, counts, N, K, **kw):
    say(f"[gmm] {form} {dtype} groups={len(counts)} rows={sum(counts)} N={N} K={K} {kw}")
    s, lhs, rhs, out = make(form, dtype, counts, N, K, **kw)
    before = out.clone()
    run(s, counts, lhs, rhs, out)
    ref, mag, n = gmm_ref(form, counts, lhs, rhs)
    rows = sum(counts)
    old = before if form == "dw" else before[:rows]
    new = out if form == "dw" else out[:rows]
    if s.accumulate:
        ref, mag = ref + old.double(), mag + old.double().abs()
    bad = (new.double() - ref).abs() > sum_bound(mag, n, ref, out.dtype)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values are off"
    if form != "dw":  # rows behind the last group stay as they were
        assert torch.equal(out[rows:], before[rows:])
    return out


FORMS = ("fwd", "dx", "dw")
RAGGED = [0, 1, 63, 64, 65, 0, 257, 5, 128, 0]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("N,K", [(64, 128), (96, 72), (1, 1), (37, 53), (8, 8), (264, 200), (130, 514)])
def test_sizes(form, dtype, out, N, K):
    check(form, dtype, RAGGED, N, K, out=out, spare=3)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("counts", [[1], [0], [0, 0, 0], [1] * 40, [300], [0] * 7 + [33], [33] + [0] * 7])
def test_counts(form, counts):
    check(form, "bf16", counts, 136, 192, spare=2)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["same", "f32"])
def test_accumulate(form, dtype, out):
    check(form, dtype, RAGGED, 72, 136, out=dtype if out == "same" else out, accumulate=True, spare=1)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lda,ldc", [(160, 104), (131, 97), (136, 73)])
def test_row_strides(form, dtype, lda, ldc):
    check(form, dtype, RAGGED, 72, 128, lda=lda, ldc=ldc, spare=4)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_split_reduction(form, dtype, out, accumulate):
    # few tiles and a long reduction
    counts, N, K = ([1999, 2100], 40, 56) if form == "dw" else ([3, 20], 48, 2056)
    if form == "dx":
        N, K = K, N
    s = make(form, dtype, counts, N, K, out=out)[0]
    assert T.moe_grouped_matmul_workspace_bytes(s) > 0
    check(form, dtype, counts, N, K, out=out, accumulate=accumulate, spare=7)


@pytest.mark.parametrize("form", FORMS)
def test_many_rows_and_tiles(form):
    check(form, "bf16", [700, 0, 1300, 256, 511, 1], 520, 776)


def ragged(groups, mean, seed=3):
    """Row counts around a mean, every seventh group empty."""
    g = torch.Generator().manual_seed(seed)
    c = torch.randint(0, 2 * mean, (groups,), generator=g)
    c[::7] = 0
    return c.tolist()


@pytest.mark.parametrize("out,accumulate", [("bf16", False), ("f32", True), ("bf16", True)])
@pytest.mark.parametrize("form,groups,mean,N,K", [
    # the tile shapes' ranges: rows per group, and enough tiles for all CUs
    ("fwd", 40, 30, 1112, 264), ("fwd", 40, 90, 1112, 264), ("fwd", 60, 200, 2056, 328),
    ("dx", 40, 25, 264, 1112), ("dx", 48, 80, 264, 2056), ("dx", 60, 200, 328, 2056),
    ("dw", 40, 50, 776, 1032), ("dw", 24, 150, 1032, 1288), ("dw", 9, 700, 264, 520),
])
def test_tile_shapes(form, groups, mean, N, K, out, accumulate):
    check(form, "bf16", ragged(groups, mean), N, K, out=out, accumulate=accumulate, spare=9)


@pytest.mark.parametrize("form,rows,N,K", [
    # more than 64 tiles for a workgroup: the tile list is made anew
    ("fwd", 1, 5120, 8), ("dx", 1, 8, 5120), ("dx", 50, 8, 4352), ("fwd", 128, 4352, 8),
])
def test_many_tiles_per_workgroup(form, rows, N, K):
    check(form, "bf16", [rows] * 1024, N, K)


@pytest.mark.parametrize("form", FORMS)
def test_most_groups(form):
    counts = [(i * 7) % 5 for i in range(1024)]
    check(form, "bf16", counts, 64, 72)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_neighbours_do_not_leak(form, dtype):
    # NaN in rows of other groups, behind the last group, and in the gap
    # between a row's end and the next row
    counts = [5, 70, 0, 33]
    s, lhs, rhs, out = make(form, dtype, counts, 72, 104, lda=112, ldc=80, spare=6)
    rows = sum(counts)
    lhs[rows:] = float("nan")
    lhs[:5] = float("nan")
    if form == "dw":
        rhs[rows:] = float("nan")
        rhs[:5] = float("nan")
    else:
        rhs[0] = float("nan")
        rhs[2] = float("inf")
    for t in (lhs, rhs, out):
        if t.dim() == 2:  # the gap
            whole = torch.as_strided(t, (t.shape[0] - 1, t.stride(0) - t.shape[1]), (t.stride(0), 1),
                                     t.storage_offset() + t.shape[1])
            whole.fill_(float("nan"))
    run(s, counts, lhs, rhs, out)
    ref, mag, n = gmm_ref(form, counts, lhs, rhs)
    part = slice(1, None) if form == "dw" else slice(5, None)
    new = (out if form == "dw" else out[:rows])[part]
    assert torch.isfinite(new).all()
    bad = (new.double() - ref[part]).abs() > sum_bound(mag[part], n, ref[part], out.dtype)
    assert not bad.any()


def test_no_rows_at_all():
    s, lhs, rhs, out = make("dw", "bf16", [0, 0], 24, 40)
    run(s, [0, 0], lhs, rhs, out)
    assert (out == 0).all()
    s, lhs, rhs, out = make("fwd", "bf16", [0, 0], 24, 40)
    run(s, [0, 0], lhs, rhs, out)
    s, lhs, rhs, out = make("dw", "f32", [0, 0], 24, 40, accumulate=True)
    before = out.clone()
    run(s, [0, 0], lhs, rhs, out)
    assert torch.equal(out, before)


@pytest.mark.parametrize("form", FORMS)
def test_offsets_outside_the_rows_stay_inside(form):
    # wrong offsets give wrong values, and touch nothing but out
    s, lhs, rhs, out = make(form, "bf16", [40, 24], 72, 64)
    ws = torch.empty(T.moe_grouped_matmul_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    for wrong in ([0, 1 << 30, (1 << 31) - 1], [-5, 70, 20], [64, 0, 64]):
        off = torch.tensor(wrong, dtype=torch.int32, device="cuda")
        T.moe_grouped_matmul(s, off, lhs, rhs, out, ws)
        torch.cuda.synchronize()


@pytest.mark.parametrize("form", FORMS)
def test_same_bits_on_another_stream_and_in_a_graph(form):
    counts, N, K = ([1999, 2100], 40, 56) if form == "dw" else ([300, 0, 21], 136, 264)
    s, lhs, rhs, out = make(form, "bf16", counts, N, K)
    run(s, counts, lhs, rhs, out)
    want = out.clone()
    off = offsets_of(counts)
    ws = torch.empty(T.moe_grouped_matmul_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    T.moe_grouped_matmul(s, off, lhs, rhs, out, ws, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        T.moe_grouped_matmul(s, off, lhs, rhs, out, ws)
    for k in range(3):
        out.zero_()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), k


def near(new, ref, mag, n):
    return not ((new.double() - ref).abs() > sum_bound(mag, n, ref, new.dtype)).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS)
def test_rows_behind_32_bits(form, dtype):
    # the last group's rows lie more than 2^32 bytes (and, in a, more than
    # 2^31 elements) behind the array's start
    N, K, counts = 64, 2048, [1_100_000, 50]
    if dtype == "f32" and form == "dw":
        counts = [0, 50]                # the first group is long enough in bf16
    dt, dev = DT[dtype], "cuda"
    M = 1_100_050
    off = offsets_of(counts) if counts[0] else torch.tensor([0, M - 50, M], dtype=torch.int32, device=dev)
    a = torch.zeros((M, K), dtype=dt, device=dev)
    c = torch.zeros((M, N), dtype=dt, device=dev)
    w = torch.randn((2, N, K), device=dev).to(dt)
    a[-60:], c[-60:] = torch.randn((60, K), device=dev).to(dt), torch.randn((60, N), device=dev).to(dt)
    s = T.make_gmm_shape(form, dtype, 2, M, N, K)
    lhs, rhs, out = {"fwd": (a, w, c), "dx": (c, w, a), "dw": (c, a, w)}[form]
    ra, rc = a[-60:].clone(), c[-60:].clone()
    ws = torch.empty(T.moe_grouped_matmul_workspace_bytes(s), dtype=torch.uint8, device=dev)
    T.moe_grouped_matmul(s, off, lhs, rhs, out, ws)
    torch.cuda.synchronize()
    if form == "dw":
        ref, mag, n = gmm_ref(form, [10, 50], rc, ra)
        assert near(out[1], ref[1], mag[1], 50)
        if counts[0]:
            assert near(out[0], ref[0], mag[0], 64)     # zeros but for ten rows
    else:
        ref, mag, n = gmm_ref(form, [10, 50], ra if form == "fwd" else rc, w)
        assert near(out[-60:], ref, mag, n)
        assert not out[:1000].any()


@pytest.mark.parametrize("form", FORMS)
def test_weights_behind_32_bits(form):
    G, N, K = 1024, 1544, 1400            # 2.2e9 elements
    counts = [0] * (G - 3) + [40, 0, 25]
    s, lhs, rhs, out = make(form, "bf16", [65], N, K)
    s.n_groups = G
    w = torch.zeros((G, N, K), dtype=torch.bfloat16, device="cuda")
    if form != "dw":
        w[-3:] = torch.randn((3, N, K), device="cuda").bfloat16()
        rhs = w
    else:
        w.fill_(5.0)
        out = w
    run(s, counts, lhs, rhs, out)
    ref, mag, n = gmm_ref(form, counts[-3:], lhs, rhs[-3:] if form != "dw" else rhs)
    assert near(out[-3:] if form == "dw" else out, ref, mag, n)
    if form == "dw":
        assert not out[: G - 3].any() and not out[G - 2].any()


def test_two_streams_at_once():
    jobs = []
    for seed, form in enumerate(("fwd", "dw", "dx", "dw")):
        counts, N, K = ([1999, 2100], 40, 56) if seed == 3 else (ragged(30, 90, seed), 264, 520)
        s, lhs, rhs, out = make(form, "bf16", counts, N, K, seed=seed)
        ws = torch.empty(T.moe_grouped_matmul_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        jobs.append((s, offsets_of(counts), lhs, rhs, out, ws))
    want = []
    for j in jobs:
        T.moe_grouped_matmul(*j)
        torch.cuda.synchronize()
        want.append(j[4].clone())
        j[4].zero_()
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        for j, st in zip(jobs, streams):
            T.moe_grouped_matmul(*j, stream=st)
    torch.cuda.synchronize()
    for j, w in zip(jobs, want):
        assert torch.equal(j[4], w)


def test_refusals():
    s, lhs, rhs, out = make("fwd", "bf16", [40, 24], 72, 64)
    off = offsets_of([40, 24])
    with pytest.raises(ValueError, match="lhs"):
        T.moe_grouped_matmul(s, off, lhs.float(), rhs, out)
    with pytest.raises(ValueError, match="lhs"):
        T.moe_grouped_matmul(s, off, lhs.t().contiguous().t(), rhs, out)
    with pytest.raises(ValueError, match="rhs"):
        T.moe_grouped_matmul(s, off, lhs, rhs[:1], out)
    with pytest.raises(ValueError, match="out"):
        T.moe_grouped_matmul(s, off, lhs, rhs, out[:10])
    with pytest.raises(ValueError, match="rhs"):
        T.moe_grouped_matmul(s, off, lhs, rhs.cpu(), out)
    split = T.make_gmm_shape("fwd", "bf16", 2, 23, 48, 2056)
    args = [torch.zeros(sh, dtype=torch.bfloat16, device="cuda") for sh in ((23, 2056), (2, 48, 2056), (23, 48))]
    with pytest.raises(ValueError, match="ws"):
        T.moe_grouped_matmul(split, offsets_of([3, 20]), *args)
    bad = torch.empty(lhs.numel() + 8, dtype=lhs.dtype, device="cuda")[1:1 + lhs.numel()].view_as(lhs)
    with pytest.raises(B.MoeError, match="EALIGN"):
        T.moe_grouped_matmul(s, off, bad, rhs, out)
