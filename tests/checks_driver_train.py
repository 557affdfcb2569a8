"""Runs the training operators through the library that MOE_MI355X_LIB names
(the debug build with device-side index-range checks, in a process of its own)
and prints one JSON line: the check bits after the valid cases, a digest of
each valid case's outputs, and the bits after each kind of wrong routing array
(the kernels keep every row inside the arrays in both builds, so nothing is
accessed out of range).

    MOE_MI355X_LIB=.../libmoe_mi355x_checks.so python -m tests.checks_driver_train
"""

import json
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

from sparse_moe_layer_03_amd import binding as B  # noqa: E402
from sparse_moe_layer_03_amd import train as T  # noqa: E402
from tests.checks_driver import digest  # noqa: E402
from tests.test_gpu_gmm import make, run  # noqa: E402
from tests.test_gpu_layer_backward import Case  # noqa: E402

# a grouped product per form on the bf16 kernels, the general kernel, and a
# split reduction
GMM = [(f, dt, counts, N, K) for f in ("fwd", "dx", "dw")
       for dt, counts, N, K in (("bf16", [0, 300, 5, 70], 136, 264), ("f32", [9, 0, 130], 72, 40),
                                ("bf16", [33, 50], 37, 53))] + [
    ("fwd", "bf16", [3, 20], 48, 2056), ("dw", "f32", [1999, 2100], 40, 56)]
LAYERS = [("bf16", 600, 128, 12, 6, 192, 4, 1.0, 1.0), ("f32", 70, 64, 5, 2, 64, 3, 1.0, 1.0)]
GRADS = ("dx", "dgate", "dlogits", "dw_router", "dw_gate", "dw_up", "dw_down")


def gmm_case(form, dtype, counts, N, K):
    s, lhs, rhs, out = make(form, dtype, counts, N, K, spare=3)
    run(s, counts, lhs, rhs, out)
    return digest(out)


def layer_case(case):
    tb = Case(*case).backward()
    return [digest(getattr(tb, n)) for n in GRADS]


def wrong_offsets(form, dtype, off):
    s, lhs, rhs, out = make(form, dtype, [40, 24], 72, 64)
    ws = torch.empty(T.moe_grouped_matmul_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    T.moe_grouped_matmul(s, torch.tensor(off, dtype=torch.int32, device="cuda"), lhs, rhs, out, ws)
    torch.cuda.synchronize()


def main():
    assert torch.cuda.is_available()
    B.moe_debug_checks(clear=True)
    out = {"lib": os.path.basename(B.LIB_PATH), "gmm": [], "layer": [], "wrong": {}}
    for c in GMM:
        out["gmm"].append(gmm_case(*c))
        print(f"[checks] {c}", file=sys.stderr, flush=True)
    for c in LAYERS:
        out["layer"].append(layer_case(c))
        print(f"[checks] {c}", file=sys.stderr, flush=True)
    out["valid_bits"] = B.moe_debug_checks(clear=True)
    for form in ("fwd", "dx", "dw"):
        for dtype in ("bf16", "f32"):
            for off in ([0, 1 << 30, (1 << 31) - 1], [-5, 40, 64], [0, 40, 20], [64, 0, 64]):
                wrong_offsets(form, dtype, off)
                out["wrong"][f"offsets {form} {dtype} {off}"] = B.moe_debug_checks(clear=True)
    c = Case(*LAYERS[1])
    for name, bad in (("perm", 1 << 30), ("perm", -1), ("inv_perm", 1 << 30), ("topk_idx", 99), ("topk_idx", -3),
                      ("offsets", 1 << 30)):
        t = getattr(c.buf, name)
        kept = t.clone()
        t[:1] = bad
        c.backward()
        t.copy_(kept)
        out["wrong"][f"{name} {bad}"] = B.moe_debug_checks(clear=True)
    print(json.dumps(out), flush=True)


if __name__ == "__main__":
    main()
