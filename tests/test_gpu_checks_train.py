"""The debug build's index-range checks in the training operators: no check
fails on valid routing arrays and the outputs are bit-identical to the release
build's; each kind of wrong routing array sets its bit.  The checks build runs
in a process of its own (tests/checks_driver_train.py)."""

import json
import os
import subprocess
import sys

import pytest

from sparse_moe_layer_03_amd import binding as B
from tests import checks_driver_train as D

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIT = {n: b for b, n in B.CHECK_BITS.items()}
# the bit that must be set; others may be too (an expert id below 0 counts as an
# FFN expert, whose slot has a row of its own)
WANT = {"perm": "MOE_CHECK_GEMM_ROW", "inv_perm": "MOE_CHECK_COMBINE_ROW", "topk_idx": "MOE_CHECK_DISPATCH_ID",
        "offsets": "MOE_CHECK_GMM_OFFSETS"}


def test_debug_checks_in_the_training_operators():
    assert os.path.exists(B.LIB_CHECKS_PATH), "build it with build(checks=True)"
    env = dict(os.environ, MOE_MI355X_LIB=B.LIB_CHECKS_PATH)
    p = subprocess.run([sys.executable, "-m", "tests.checks_driver_train"], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=200)
    assert p.returncode == 0, p.stderr[-3000:]
    res = json.loads(p.stdout.strip().splitlines()[-1])
    print(res, flush=True)
    assert res["lib"] == os.path.basename(B.LIB_CHECKS_PATH)
    assert res["valid_bits"] == 0, [n for b, n in B.CHECK_BITS.items() if res["valid_bits"] & b]
    assert len(res["wrong"]) == 30
    for name, bits in res["wrong"].items():
        assert bits & BIT[WANT[name.split()[0]]], (name, bits)
    # the release build (this process) computes the same bits
    assert [D.gmm_case(*c) for c in D.GMM] == res["gmm"]
    assert [D.layer_case(c) for c in D.LAYERS] == res["layer"]
