"""Build libttt.so (the HIP library behind include/ttt.h) in-tree for gfx950."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libttt.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Wall", "-Wno-unused-command-line-argument",
    # no packed-fp32 instructions in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in ordinary VGPRs: the state and the accumulators feed VALU
    # work every step, and AGPR destinations would add a copy for each value
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    f"-I{os.path.join(ROOT, 'include')}",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    msg = "\n".join(l for l in (res.stdout + res.stderr).splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{msg}")
    if verbose and msg.strip():
        print(msg, file=sys.stderr)


def build(verbose: bool = False, extra=()) -> str:
    """Compile every source to an object of its own (as many at a time as there
    are CPUs, at most 8) and link them; the library is replaced at the end."""
    tmp = LIB + ".tmp"
    objects = tempfile.mkdtemp(prefix="libttt_")
    try:
        flags = [f for f in FLAGS if f != "-shared"]
        outs = [os.path.join(objects, os.path.basename(src)[:-4] + ".o") for src in sources()]
        with ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            list(pool.map(lambda p: _run([HIPCC, *flags, *extra, "-c", "-o", p[1], p[0]], verbose),
                          zip(sources(), outs)))
        _run([HIPCC, *FLAGS, *extra, "-o", tmp, *outs], verbose)
    finally:
        shutil.rmtree(objects, ignore_errors=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
