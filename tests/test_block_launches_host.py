"""The launches of the operators around the layer over the sizes that
moe_block.h allows, recorded on the CPU as in tests/test_train_launches_host.py:
a call that its checks accept must not fail in the middle of its launches for
their size.  And the binding's refusal of a stream of another device."""

import ctypes
import json
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# T, E, groups, kept
SELECT = [(1, 1, 1, 1), (128, 768, 1, 1), ((1 << 27) - 1, 1024, 64, 33), ((1 << 27) - 1, 1023, 33, 32), ((1 << 27) - 1, 8, 2, 1)]
QUANT = [(1, 1), ((1 << 27) - 1, 131071), ((1 << 27) - 1, 64), (0, 8)]
# groups, M, N, K
PRODUCT = [(1, 1, 1, 1), (1, (1 << 27) - 1, 1 << 20, 131071), (1024, (1 << 27) - 1, 1 << 20, 131056), (7, 0, 64, 64), (1, 3, 64, 131056),
           (1024, 5, 1 << 20, 15)]
# T, d, n, z, f, k
FFN = [(1, 64, 1, 0, 64, 1), ((1 << 25) - 1025, 64, 3, 0, 64, 3), (16380, 131008, 700, 300, 131008, 16)]
# T, d, tokens a gate row
NORM = [(1, 1, 1), ((1 << 27) - 1, 32768, 1), ((1 << 27) - 1, 1, (1 << 31) - 1), ((1 << 27) - 1, 32761, 3), (0, 64, 1)]


def record():
    """In the process of its own: one JSON line, [case, status, launches] each."""
    sys.path.insert(0, ROOT)
    from sparse_moe_layer_03_amd import binding as B
    from sparse_moe_layer_03_amd import block as K
    P, ref, log, out = ctypes.c_void_p, ctypes.byref, os.environ["LAUNCH_LOG"], []
    at = [(i + 1) << 56 for i in range(16)]         # addresses that are never followed, far apart

    def case(name, call):
        open(log, "w").close()
        rc = call()
        out.append([name, rc, [[int(v) for v in line.split()] for line in open(log)]])

    for T, E, G, kept in SELECT:
        s, p = B.make_shape(T, 64, E, 0, 64, 1, "f32"), K.make_select("softmax", G, kept)
        case(["select", T, E, G], lambda: K.lib().moe_select(ref(s), ref(p), P(at[0]), E, *map(P, at[1:4]), None))
        case(["select_backward", T, E, G], lambda: K.lib().moe_select_backward(ref(s), ref(p), P(at[0]), E, *map(P, at[1:4]), None))
    for M, k in QUANT:
        for dt in ("bf16", "f32"):
            s = K.make_quant_shape(dt, M, k)
            case(["quantize", M, k], lambda: K.lib().moe_quantize_rows(ref(s), *map(P, at[:3]), None))
    for G, M, N, k in PRODUCT:
        for dt in ("bf16", "f32"):
            s = K.make_i8_shape(dt, G, M, N, k)
            case(["matmul", M, G, N, k], lambda: K.lib().moe_matmul_i8(ref(s), *map(P, at[:7]), None))
    for c in FFN:
        for dt in ("bf16", "f32"):
            s = B.make_shape(*c, dt)
            assert K.moe_expert_ffn_i8_workspace_bytes(s) > 0
            io = K.MoeFfnI8IO(*at[:12])
            io.xq = io.x_scale = None
            case(["ffn", *c], lambda: K.lib().moe_expert_ffn_i8(ref(s), ref(io), P(at[12]), None))
    for T, d, per in NORM:
        for dt in ("bf16", "f32"):
            s = K.make_norm_shape(T, d, dt, 1e-6, 1.0, per)
            a = iter(at)
            m = lambda: (next(a), d)  # noqa: E731
            io = K.MoeNormIO(*m(), *m(), next(a), next(a), next(a), *m(), *m(), next(a), next(a))
            case(["norm", T, d], lambda: K.lib().moe_norm_residual(ref(s), ref(io), None))
            a = iter(at)
            io = K.MoeNormGradIO(*m(), *m(), next(a), next(a), next(a), *m(), *m(), *m(), *m(), next(a), next(a), next(a), 0, 0)
            assert K.moe_norm_residual_backward_workspace_bytes(s) > 0
            case(["norm_backward", T, d], lambda: K.lib().moe_norm_residual_backward(ref(s), ref(io), P(at[13]), None))
    print(json.dumps(out))


@pytest.fixture(scope="module")
def recorded(tmp_path_factory):
    d = tmp_path_factory.mktemp("launches")
    so = str(d / "recorder.so")
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", os.path.join(ROOT, "tests", "launch_recorder.c"), "-o", so],
                   check=True)
    env = dict(os.environ, LAUNCH_LOG=str(d / "log"), LD_PRELOAD=so)
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


def test_every_accepted_size_can_be_launched(recorded):
    assert len(recorded) == 2 * len(SELECT) + 2 * (len(QUANT) + len(PRODUCT) + len(FFN) + 2 * len(NORM))
    for name, rc, launches in recorded:
        assert rc == 0, (name, rc)
        assert launches or name[1] == 0, name       # (no rows: nothing to launch)
        for grid, block, ok in launches:
            assert 0 < grid and grid * block < 1 << 32 and ok, (name, grid, block)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    from sparse_moe_layer_03_amd import block as K

    class Stream:
        def __init__(self, device):
            self.device, self.cuda_stream = torch.device(device), 64

    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    calls = []

    class Lib:
        def moe_select(self, *args):
            calls.append(args)
            return 0

    monkeypatch.setattr(K, "lib", lambda: Lib())
    with pytest.raises(ValueError, match="stream: on cuda:1, needed on cuda:0"):
        K._run("moe_select", 0, Stream("cuda:1"), 7)
    assert not calls
    K._run("moe_select", 0, Stream("cuda:0"), 7)
    assert calls == [(7, 64)]


if __name__ == "__main__":
    record()
