"""The launches of the training operators over the sizes that moe_train.h
allows, recorded on the CPU: tests/launch_recorder.c stands in for the HIP
runtime's launch calls in a process of its own, so nothing is computed and no
memory is touched.  A launch holds fewer than 2^32 threads; a call that its
checks accept must not fail in the middle of its launches for their size."""

import ctypes
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (T, d_model, n_ffn, n_zero, d_ff, top_k, dtype): up to T * top_k = 2^27 - 1
BACKWARD = [(64, 128, 8, 4, 256, 2, "f32"), (4096, 2048, 64, 32, 1024, 8, "bf16")] + [
    (T, 64, 14, 2, 64, k, dt) for dt in ("bf16", "f32")
    for T, k in (((1 << 24) - 1, 1), (1 << 24, 1), ((1 << 23) + 1, 2), ((1 << 27) - 1, 1), ((1 << 23) - 1, 16))]
# (form, dtype, groups, M, N, K)
GMM = [(f, dt, g, (1 << 27) - 1, n, k) for f in ("fwd", "dx", "dw") for dt in ("bf16", "f32")
       for g, n, k in ((1, 8, 8), (1024, 64, 64), (7, 1 << 20, 8), (7, 8, 1 << 20), (3, 129, 257))]


def record():
    """In the process of its own: one JSON line, [case, status, launches] each."""
    sys.path.insert(0, ROOT)
    from sparse_moe_layer_03_amd import binding as B
    from sparse_moe_layer_03_amd import train as T
    A, P, log, out = 0x1000, ctypes.c_void_p, os.environ["LAUNCH_LOG"], []

    def case(name, call):
        open(log, "w").close()
        rc = call()
        out.append([name, rc, [[int(v) for v in line.split()] for line in open(log)]])

    for c in BACKWARD:
        for router in (True, False):
            io = T.MoeBackwardIO(*[A] * len(T._IO_IN + T._IO_OUT), 0, 0)
            if not router:
                io.w_router = io.logits = io.dlogits = io.dw_router = None
            s = B.make_shape(*c)
            assert T.moe_layer_backward_workspace_bytes(s) > 0
            case(["backward", *c, router],
                 lambda: T.lib().moe_layer_backward(ctypes.byref(s), ctypes.byref(io), P(A), None))
    for form, dt, g, M, N, K in GMM:
        s = T.make_gmm_shape(form, dt, g, M, N, K)
        case([form, dt, g, M, N, K],
             lambda: T.lib().moe_grouped_matmul(ctypes.byref(s), *[P(A)] * 5, None))
    for n, count in ((0, 1), (1 << 40, 1), (1, 200)):
        arr = (T.MoeAdamwTensor * count)(*[T.MoeAdamwTensor(A, A, None, A, A, A, A, n, 0, 0, 0.0)] * count)
        p = T.make_adamw_params(1e-3)
        case(["adamw", n, count],
             lambda: T.lib().moe_adamw(ctypes.byref(p), arr, count, P(A), None, None, None))
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
    assert len(recorded) == 2 * len(BACKWARD) + len(GMM) + 3
    for name, rc, launches in recorded:
        assert launches, name
        for grid, block, ok in launches:
            assert 0 < grid and grid * block < 1 << 32 and ok, (name, grid, block)
        assert rc == 0, (name, rc)


def test_a_call_launches_what_its_shape_needs(recorded):
    # the same launches whatever the number of rows
    count = {}
    for name, _, launches in recorded:
        if name[0] == "backward":
            count.setdefault((name[7], name[8]), set()).add(len(launches))
    assert all(len(v) == 1 for v in count.values()), count


if __name__ == "__main__":
    record()
