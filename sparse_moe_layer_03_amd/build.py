"""Builds libmoe_mi355x.so (the C-ABI library) and its debug build with
device-side index-range checks, libmoe_mi355x_checks.so, in-tree with hipcc
for gfx950.

    python -m sparse_moe_layer_03_amd.build [--release-only]
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_mi355x.so")
# debug build with the device-side index-range checks (moe_debug_checks)
LIB_CHECKS = os.path.join(PKG, "libmoe_mi355x_checks.so")
OBJ_CHECKS = os.path.join(PKG, "_build_checks")
ARCH = "gfx950"

SOURCES = ["api.hip", "gemm.hip", "gemm_big.hip", "route.hip", "dispatch.hip", "combine.hip", "pid.hip",
           "noalloc.hip", "eplb.hip", "train_api.hip", "gmm_general.hip",
           "gmm_mfma.hip", "layer_bwd.hip", "adamw.hip", "block_api.hip", "select.hip", "norm.hip",
           "quant.hip", "gmm_i8.hip", "i8_general.hip"]

# Integer accumulators that leave the reduction's loop at several places are
# taken apart into single registers by default, and copied at each of them
# (256 x 256 tiles: 1500 spilled registers instead of a few).
FILE_FLAGS = {"gmm_i8.hip": ["-mllvm", "-amdgpu-codegenprepare-break-large-phis=false"]}

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # packed fp32 VALU forms stay disabled on this target
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fno-gpu-rdc", "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
    f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
]


# Checking build for host-side tests: AddressSanitizer and
# UndefinedBehaviorSanitizer on the host code only (argument checks,
# planning, launch set-up; each flag behind -Xarch_host, the device code is
# built as usual).  The sanitizer runtime is resolved when the library is
# loaded (LD_PRELOAD of the runtime), so the link line needs no flag.
SANITIZE_FLAGS = ["-O1", "-g", "-Xarch_host", "-fno-omit-frame-pointer",
                  "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                  "-Xarch_host", "-fno-sanitize-recover=undefined"]


def _compile(src: str, obj_dir: str = OBJ, extra=()) -> str:
    obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
    flags = [f for f in CFLAGS if not (any(x.startswith("-O") for x in extra) and f == "-O3")]
    cmd = [HIPCC, *flags, *FILE_FLAGS.get(src, ()), *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{p.stdout}\n{p.stderr}")
    return obj


def build(verbose: bool = False, sanitize_out: str = "", checks: bool = False) -> str:
    """Builds the library in-tree; with sanitize_out, builds the host-side
    sanitizer build to that path instead; with checks, the debug build with
    the device-side index-range checks (LIB_CHECKS)."""
    if sanitize_out:
        obj_dir, extra, lib = os.path.join(os.path.dirname(sanitize_out), "_obj"), SANITIZE_FLAGS, \
            sanitize_out
    elif checks:
        obj_dir, extra, lib = OBJ_CHECKS, ["-DMOE_DEVICE_CHECKS"], LIB_CHECKS
    else:
        obj_dir, extra, lib = OBJ, (), LIB
    os.makedirs(obj_dir, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(6, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, obj_dir, extra), SOURCES))
    tmp = lib + ".tmp"
    link = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}"]
    p = subprocess.run([*link, *objs, "-o", tmp], capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, lib)
    if verbose:
        print(f"built {lib}")
    return lib


if __name__ == "__main__":
    build(verbose=True)
    if "--release-only" not in sys.argv[1:]:
        build(verbose=True, checks=True)
    sys.exit(0)
