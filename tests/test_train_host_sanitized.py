"""The training operators' host checks again, against a build of the library
whose host code carries AddressSanitizer and UndefinedBehaviorSanitizer, as
tests/test_abi_host_sanitized.py does for the layer's."""

import os
import subprocess
import sys
import tempfile

import pytest

from tests.test_abi_host_sanitized import ROOT, _asan_runtime


@pytest.mark.skipif(_asan_runtime() is None, reason="no clang AddressSanitizer runtime found")
def test_train_host_checks_under_address_and_ub_sanitizers():
    from sparse_moe_layer_03_amd import build as Bld
    d = tempfile.mkdtemp(prefix="moe_san_")
    lib = Bld.build(sanitize_out=os.path.join(d, "libmoe_san.so"))
    env = dict(os.environ, MOE_MI355X_LIB=lib, LD_PRELOAD=_asan_runtime(),
               ASAN_OPTIONS="detect_leaks=0:halt_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.join(ROOT, "tests", "test_train_host.py"), "-k", "not struct_sizes"],
                       cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    out = r.stdout + r.stderr
    assert r.returncode == 0, out[-3000:]
    assert "AddressSanitizer" not in out and "runtime error" not in out, out[-3000:]
    assert " passed" in out
