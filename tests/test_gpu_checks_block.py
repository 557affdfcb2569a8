"""The debug build's index-range checks in the operators around the layer: no
check fails on valid routing arrays and the outputs are bit-identical to the
release build's; each kind of wrong routing array sets its bit.  The checks
build runs in a process of its own (tests/checks_driver_block.py)."""

import json
import os
import subprocess
import sys

import pytest

from sparse_moe_layer_03_amd import binding as B
from tests import checks_driver_block as D

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BIT = {n: b for b, n in B.CHECK_BITS.items()}
WANT = {"perm": "MOE_CHECK_GEMM_ROW", "topk_idx": "MOE_CHECK_DISPATCH_ID", "offsets": "MOE_CHECK_GMM_OFFSETS"}


def test_debug_checks_in_the_operators_around_the_layer():
    assert os.path.exists(B.LIB_CHECKS_PATH), "build it with build(checks=True)"
    env = dict(os.environ, MOE_MI355X_LIB=B.LIB_CHECKS_PATH)
    p = subprocess.run([sys.executable, "-m", "tests.checks_driver_block"], cwd=ROOT, env=env, capture_output=True,
                       text=True, timeout=100)
    assert p.returncode == 0, p.stderr[-3000:]
    res = json.loads(p.stdout.strip().splitlines()[-1])
    assert res["lib"] == os.path.basename(B.LIB_CHECKS_PATH)
    assert res["valid_bits"] == 0, [n for b, n in B.CHECK_BITS.items() if res["valid_bits"] & b]
    assert len(res["wrong"]) == 13
    for name, bits in res["wrong"].items():
        assert bits & BIT[WANT[name.split()[0]]], (name, bits)
    # the release build (this process) computes the same bits
    assert [D.product(*c) for c in D.PRODUCTS] == res["products"]
    assert [D.ffn(c) for c in D.FFNS] == res["ffn"]
    assert [D.model(*c) for c in D.MODELS] == res["models"]
