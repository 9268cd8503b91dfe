"""Builds libsgemm.so (the HIP kernels and the C ABI) and libsgemm_probe.so
(the benchmark's clock probe) for gfx950 with hipcc.  The library's source
files are compiled side by side and linked.

``python -m tiled_fp32_gemm_amd.build [--asm]`` compiles in-tree; ``--asm``
also writes the device assembly next to the sources' build folder
(``_build/``) for instruction counts.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libsgemm.so")
PROBE_LIB = os.path.join(HERE, "libsgemm_probe.so")
ROOT = os.path.dirname(HERE)
ASM_DIR = os.path.join(ROOT, "_build")
ARCH = "gfx950"
JOBS = 8     # compilations at once

# Packed FP32 instructions are kept out of the generated code (the vector
# kernels use single fused multiply-adds; the matrix kernels do not need them).
DEVICE_FLAGS = ["--offload-arch=" + ARCH, "-O3", "-std=c++17",
                "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                "-ffp-contract=fast", "-Wall"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) +
                  glob.glob(os.path.join(CSRC, "*.hpp")) +
                  glob.glob(os.path.join(ROOT, "include", "*.h")))


def library_sources() -> list[str]:
    """The sources of libsgemm.so, the longest to compile first."""
    names = sorted(glob.glob(os.path.join(CSRC, "*.hip")), key=os.path.getsize, reverse=True)
    return [n for n in names if os.path.basename(n) != "probe.hip"]


def _hipcc(args: list[str], out: str, verbose: bool) -> str:
    tmp = out + f".tmp{os.getpid()}"
    cmd = ["hipcc", *DEVICE_FLAGS, "-fPIC", *args, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


def build(verbose: bool = False) -> str:
    """Compile the sources under ``csrc`` into ``libsgemm.so`` and
    ``csrc/probe.hip`` into ``libsgemm_probe.so`` (always recompiles)."""
    link = ["-shared", "-Wl,-rpath,/opt/rocm/lib"]
    with tempfile.TemporaryDirectory() as objects, \
            concurrent.futures.ThreadPoolExecutor(JOBS) as pool:
        jobs = [pool.submit(_hipcc, ["-c", src], os.path.join(
            objects, os.path.basename(src) + ".o"), verbose) for src in library_sources()]
        probe = pool.submit(_hipcc, [*link, os.path.join(CSRC, "probe.hip")], PROBE_LIB, verbose)
        probe.result()
        return _hipcc([*link, *(j.result() for j in jobs)], LIB, verbose)


def build_asm() -> str:
    """Device assembly of the library, for reading our own instruction mix."""
    os.makedirs(ASM_DIR, exist_ok=True)
    out = os.path.join(ASM_DIR, f"sgemm-{ARCH}.s")
    cmd = ["hipcc", *DEVICE_FLAGS, "--offload-device-only", "-S",
           os.path.join(CSRC, "sgemm.hip"), "-o", out]
    subprocess.run(cmd, check=True)
    return out


def ensure_built() -> str:
    """Build only when a library is missing or older than a source."""
    newest = max(os.path.getmtime(s) for s in sources())
    if any(not os.path.exists(p) or os.path.getmtime(p) < newest
           for p in (LIB, PROBE_LIB)):
        return build()
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
    if "--asm" in sys.argv:
        print(build_asm())
