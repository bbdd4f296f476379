"""Build libfq.so (all HIP sources of csrc/) for gfx950 with hipcc, and the native
call marshalling _fqbind.so (bind/bind.cpp, host code) with g++, in-tree.

    python moe_fake_quant_amd/build.py          # or build() from Python

Both land next to this file; the Python binding loads them from there.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfq.so")
ARCH = "gfx950"


def hipcc() -> str:
    p = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(p):
        raise RuntimeError("hipcc not found (ROCm toolchain required to build libfq)")
    return p


def flags(extra=()):
    return [
        f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-shared",
        # codec arithmetic is specified without fused multiply-adds
        "-ffp-contract=off",
        # no packed fp32 VALU ops (v_pk_*_f32) in generated code
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        f"-I{INCLUDE}", f"-I{CSRC}",
        *extra,
    ]


def build(verbose: bool = False, extra=()) -> str:
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), *flags(extra), "-o", tmp, *srcs]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = res.stdout + res.stderr
    # hipcc's host pass does not know the packed-fp32 feature and says so
    noise = "is not a recognized feature for this target"
    lines = [ln for ln in out.splitlines() if noise not in ln]
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(lines))
    if verbose and lines:
        print("\n".join(lines))
    os.replace(tmp, LIB)
    build_bind(verbose)
    return LIB


BIND_SRC = os.path.join(HERE, "bind", "bind.cpp")
BIND_LIB = os.path.join(HERE, "_fqbind.so")


def build_bind(verbose: bool = False) -> str:
    """The native marshalling of torch tensors, linked against libfq.so beside it."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        raise RuntimeError("torch not found (its headers are needed for bind/bind.cpp)")
    torch = os.path.dirname(spec.origin)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    tmp = BIND_LIB + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM", f"-I{INCLUDE}", f"-I{torch}/include",
           f"-I{torch}/include/torch/csrc/api/include", f"-I{rocm}/include", "-I/opt/rocm/include",
           f"-I{sysconfig.get_paths()['include']}", BIND_SRC, "-o", tmp, f"-L{HERE}", "-l:libfq.so",
           "-Wl,-rpath,$ORIGIN", f"-L{torch}/lib", "-lc10", "-lc10_hip", "-ltorch_python",
           f"-Wl,-rpath,{torch}/lib"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, BIND_LIB)
    return BIND_LIB


PEAKS_SRC = os.path.join(HERE, "peaks", "peaks.hip")
PEAKS_LIB = os.path.join(HERE, "libfqpeaks.so")


def build_peaks(verbose: bool = False) -> str:
    """The benchmark's measured-peak probes (MFMA chain, device copy): a
    separate small library, not part of libfq's path."""
    tmp = PEAKS_LIB + ".tmp"
    cmd = [hipcc(), *flags(), "-o", tmp, PEAKS_SRC]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    lines = [ln for ln in (res.stdout + res.stderr).splitlines() if noise not in ln]
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(lines))
    os.replace(tmp, PEAKS_LIB)
    return PEAKS_LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
    print(LIB)
