"""Runs the operators around the layer through the library that MOE_MI355X_LIB
names (the debug build with device-side index-range checks, in a process of its
own) and prints one JSON line, as tests/checks_driver_train.py does for the
training operators: the check bits after the valid cases, a digest of each valid
case's outputs, and the bits after each kind of wrong routing array.

    MOE_MI355X_LIB=.../libmoe_mi355x_checks.so python -m tests.checks_driver_block
"""

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from sparse_moe_layer_03_amd import binding as B  # noqa: E402
from sparse_moe_layer_03_amd import block as K  # noqa: E402
from tests.block_util import codes  # noqa: E402
from tests.checks_driver import digest  # noqa: E402
from tests.test_gpu_block import RULES, Model  # noqa: E402
from tests.test_gpu_i8 import Ffn  # noqa: E402
from tests.train_util import offsets_of  # noqa: E402

# counts, N, K: the fast tiles, odd rows, a split reduction
PRODUCTS = [([0, 300, 5, 70], 136, 256), ([9, 0, 130], 72, 47), ([3, 20], 48, 6144), ([260, 1, 280], 4096, 128)]
FFNS = [(300, 128, 192, 12, 6, 4, "bf16"), (70, 64, 64, 5, 2, 3, "f32")]
MODELS = [(dt, r) for dt in ("bf16", "f32") for r in RULES]


def product(counts, N, Kn, off=None):
    g = torch.Generator(device="cuda").manual_seed(0)
    M, G = sum(counts) + 2, len(counts)
    s = K.make_i8_shape("bf16", G, M, N, Kn)
    a, w = codes((M, Kn), g), codes((G, N, Kn), g)
    one = torch.ones(max(M, G * N), device="cuda")
    out = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(K.moe_matmul_i8_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    o = offsets_of(counts) if off is None else torch.tensor(off, dtype=torch.int32, device="cuda")
    K.moe_matmul_i8(s, o, a, one, w, one, out, ws)
    torch.cuda.synchronize()
    return digest(out)


def ffn(case):
    return digest(Ffn(*case).run())


def model(dtype, rule):
    m = Model(dtype, rule)
    m.forward()
    m.prepare_backward()
    m.backward()
    torch.cuda.synchronize()
    return [digest(t) for t in (m.buf[2].layer.topk_idx, m.buf[2].r, m.buf[2].h, *m.outputs().values())]


def main():
    assert torch.cuda.is_available()
    B.moe_debug_checks(clear=True)
    out = {"lib": os.path.basename(B.LIB_PATH), "wrong": {}}
    out["products"] = [product(*c) for c in PRODUCTS]
    out["ffn"] = [ffn(c) for c in FFNS]
    out["models"] = [model(*c) for c in MODELS]
    out["valid_bits"] = B.moe_debug_checks(clear=True)
    for Kn in (64, 47):
        for off in ([0, 1 << 30, (1 << 31) - 1], [-5, 40, 64], [0, 40, 20], [64, 0, 64]):
            product([40, 24], 72, Kn, off)
            out["wrong"][f"offsets {Kn} {off}"] = B.moe_debug_checks(clear=True)
    c = Ffn(*FFNS[1])
    for bad in (1 << 30, -1):
        perm = c.perm.clone()
        perm[:1] = bad
        c.run(perm=perm)
        out["wrong"][f"perm {bad}"] = B.moe_debug_checks(clear=True)
    s, p = B.make_shape(9, 64, 12, 0, 64, 2, "f32"), K.make_select()
    for bad in (12, -1, 1 << 30):
        idx = torch.zeros((9, 2), dtype=torch.int32, device="cuda")
        idx[4, 1] = bad
        x, dg = torch.zeros((9, 12), device="cuda"), torch.ones((9, 2), device="cuda")
        K.moe_select_backward(s, p, x, idx, dg, torch.empty_like(x))
        torch.cuda.synchronize()
        out["wrong"][f"topk_idx {bad}"] = B.moe_debug_checks(clear=True)
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
