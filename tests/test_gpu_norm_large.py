"""The norms around a block on arrays beyond 32 MiB with rows of whole chunks,
which are loaded and stored non-temporally: each row length's kernel, in both
types, forward and backward, in place, with strides and codes."""

import pytest
import torch

from sparse_moe_layer_03_amd import block as K
from tests.block_util import quantise_ref
from tests.test_gpu_norm import Case

pytestmark = pytest.mark.gpu

BEYOND = 34 << 20       # bytes
WIDTHS = [64, 512, 1024, 2048, 4096, 6144, 8192, 16384, 32768]


def tokens(d, dtype):
    return BEYOND // (d * (2 if dtype == "bf16" else 4)) + 1


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", WIDTHS)
def test_large_arrays(dtype, d):
    T = tokens(d, dtype)
    c = Case(T, d, dtype, per=max(1, T // 7)).forward().check().backward().check_backward()
    c.backward(accumulate=True).check_backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(post=False), dict(pre=False), dict(gate=False), dict(x=False), dict(y=False)])
def test_parts_that_fall_out_of_large_arrays(dtype, kw):
    d = 2048
    c = Case(tokens(d, dtype), d, dtype, per=1000, **kw).forward().check()
    c.backward(dx=c.x is not None or c.y is None).check_backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,ld", [(1000, 1003), (4096, 4104)])
def test_strides_of_large_arrays(dtype, d, ld):
    Case(tokens(d, dtype), d, dtype, per=64, ld=ld).forward().check().backward().check_backward()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [512, 6144])
def test_codes_and_places_of_large_arrays(dtype, d):
    T = tokens(d, dtype)
    c = Case(T, d, dtype, per=T).forward().backward()
    q, scale = torch.empty((T, d), dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    x, h = c.x.clone(), torch.empty_like(c.h)
    c.forward(x=x, r=x, h=h, q=q, q_scale=scale)
    assert torch.equal(x, c.r) and torch.equal(h, c.h)
    wq, ws = quantise_ref(h)
    assert torch.equal(q.double(), wq) and torch.equal(scale, ws)
    new = {n: c.args[n].clone() for n in ("r", "y", "dr", "dh")}
    K.moe_norm_residual_backward(c.s, c.ws, **{**c.args, **new, "dx": new["dr"], "dy": new["y"]})
    torch.cuda.synchronize()
    assert torch.equal(new["dr"], c.out["dx"]) and torch.equal(new["y"], c.out["dy"])
