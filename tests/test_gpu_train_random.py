"""Seeded random shapes through moe_grouped_matmul and moe_layer_backward,
held to the same references and bounds as their own tests: forms, types,
strides, group counts and sizes in combinations that no list names."""

import random

import pytest
import torch

from tests.test_gpu_gmm import check
from tests.test_gpu_layer_backward import Case, TOL, far

pytestmark = pytest.mark.gpu


def log_int(r, lo, hi):
    return int(round(2 ** r.uniform(torch.tensor(float(lo)).log2().item(), torch.tensor(float(hi)).log2().item())))


@pytest.mark.parametrize("seed", range(80))
def test_grouped_matmul(seed):
    r = random.Random(seed)
    form, dtype = r.choice(["fwd", "dx", "dw"]), r.choice(["bf16", "bf16", "f32"])
    groups = log_int(r, 1, 300)
    while True:
        rows, N, K = log_int(r, 1, 6000), log_int(r, 1, 3000), log_int(r, 1, 3000)
        if r.random() < 0.7:
            N, K = max(8, N // 8 * 8), max(8, K // 8 * 8)
        if groups * N * K < 1.2e8 and rows * N * K < 4e9:
            break
    g = torch.Generator().manual_seed(seed)
    q = torch.arange(1, groups + 1, dtype=torch.float64).pow(-r.choice([0.0, 0.7, 1.5]))[torch.randperm(groups, generator=g)]
    counts = torch.bincount(torch.multinomial(q, rows, replacement=True, generator=g), minlength=groups).tolist()
    gap = r.choice([0, 0, 1, 8, 24])
    check(form, dtype, counts, N, K, spare=r.choice([0, 1, 77]), lda=K + gap, ldc=N + r.choice([0, gap]),
          out=r.choice([dtype, "f32"]), accumulate=r.random() < 0.4, seed=seed)


@pytest.mark.parametrize("seed", range(24))
def test_layer_backward(seed):
    r = random.Random(1000 + seed)
    dtype = r.choice(["bf16", "bf16", "f32"])
    n_ffn, n_zero = log_int(r, 1, 60), r.choice([0, log_int(r, 1, 40)])
    k = min(log_int(r, 1, 12), n_ffn + n_zero)
    while True:
        T, d, ff = log_int(r, 1, 1500), 64 * log_int(r, 1, 8), 64 * log_int(r, 1, 8)
        if T * k * d * ff < 1e9:
            break
    case = (dtype, T, d, n_ffn, n_zero, ff, k, r.choice([1.0, 2.5]), r.choice([0.0, 1.0, 2.0]))
    print("[layer]", case, flush=True)
    c = Case(*case, seed=seed)
    tb, ref = c.backward(), c.reference()
    for name, want in ref.items():
        assert far(getattr(tb, name), want) <= TOL[dtype], (case, name)
