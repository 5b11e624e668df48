"""Build libengram.so (the HIP kernels and the C ABI) for gfx950 with hipcc."""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libengram.so")

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared", "-Wall",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def build(verbose: bool = False) -> str:
    """Every source compiled on its own, side by side, then linked."""
    tmp = LIB + ".tmp"
    compile_flags = [f for f in HIPCC_FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as objects:
        jobs, linked = [], []
        for src in sources():
            obj = os.path.join(objects, os.path.basename(src) + ".o")
            jobs.append(["hipcc", *compile_flags, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, src])
            linked.append(obj)
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            done = list(pool.map(lambda c: (c, _run(c, verbose)), jobs))
        done.append((["link"], _run(["hipcc", "--offload-arch=gfx950", "-fPIC", "-shared", "-o", tmp, *linked], verbose)
                     if all(r.returncode == 0 for _, r in done) else None))
    noise = "is not a recognized feature for this target"
    for cmd, r in done:
        msgs = [l for l in (r.stdout + r.stderr).splitlines() if noise not in l] if r else []
        if r is None or r.returncode != 0:
            sys.stderr.write("\n".join(msgs) + "\n")
            raise RuntimeError(f"hipcc failed building {LIB}: {cmd[-1]}")
        if verbose and msgs:
            print("\n".join(msgs))
    os.replace(tmp, LIB)
    return LIB


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.run(cmd, capture_output=True, text=True)


PROBE_SRC = os.path.join(PKG, "probe", "hbm_probe.hip")
PROBE_BIN = os.path.join(PKG, "probe", "hbm_probe")
VALU_SRC = os.path.join(PKG, "probe", "valu_rate.hip")
VALU_BIN = os.path.join(PKG, "probe", "valu_rate")


def _build_program(src: str, out: str) -> str:
    tmp = out + ".tmp"
    cmd = ["hipcc", *[f for f in HIPCC_FLAGS if f not in ("-fPIC", "-shared")], "-o", tmp, src]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed ({r.returncode}) building {out}")
    os.replace(tmp, out)
    return out


def build_probe(verbose: bool = False) -> str:
    """The measurement programs (not part of libengram): the HBM streaming
    ceilings (hbm_probe) and the VALU issue costs (valu_rate)."""
    _build_program(VALU_SRC, VALU_BIN)
    return _build_program(PROBE_SRC, PROBE_BIN)


PROBE_LIB_SRC = os.path.join(PKG, "probe", "stream_lib.hip")
PROBE_LIB = os.path.join(PKG, "probe", "libengram_probe.so")


def build_probe_lib(verbose: bool = False) -> str:
    """The probe's streaming kernels as a shared library (bench.py --same-buffers)."""
    tmp = PROBE_LIB + ".tmp"
    cmd = ["hipcc", *HIPCC_FLAGS, "-o", tmp, PROBE_LIB_SRC]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed ({r.returncode}) building {PROBE_LIB}")
    os.replace(tmp, PROBE_LIB)
    return PROBE_LIB


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_probe(verbose=True))
    print(build_probe_lib(verbose=True))
