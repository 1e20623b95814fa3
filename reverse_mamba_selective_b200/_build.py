"""Build libr2l.so and libr2l_mixer.so in-tree with nvcc for sm_100a (B200).

Each library is one translation unit (csrc/r2l.cu, csrc/mixer/mixer.cu) linked against the static CUDA
runtime; the driver API (tensor-map encoding) is reached at run time through
cudaGetDriverEntryPoint, so neither .so has a link-time dependency on libcuda.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from typing import List, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libr2l.so")
MIXER_CSRC = os.path.join(CSRC, "mixer")
MIXER_LIB = os.path.join(PKG, "libr2l_mixer.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libr2l.so")


def _files(folder: str) -> List[str]:
    return sorted(os.path.join(folder, f) for f in os.listdir(folder) if f.endswith((".cu", ".cuh")))


def sources() -> List[str]:
    """What libr2l.so is built from, beside its header."""
    return _files(CSRC)


def mixer_sources() -> List[str]:
    """What libr2l_mixer.so is built from, beside its headers: its own files and the shared device helpers."""
    return _files(MIXER_CSRC) + [os.path.join(CSRC, f) for f in ("common.cuh", "tc_common.cuh", "tmap.cuh")]


def _compile(main: str, out: str, deps: List[str], force: bool, extra: Optional[List[str]], verbose: bool) -> str:
    stale = force or not os.path.exists(out) or any(os.path.getmtime(s) > os.path.getmtime(out) for s in deps)
    if not stale:
        return out
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--shared", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "-cudart", "static",
           "-I", INCLUDE, "-I", CSRC, "-o", out + ".tmp", main]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    cmd += list(extra or [])
    subprocess.check_call(cmd)
    os.replace(out + ".tmp", out)
    return out


def build_mixer(force: bool = False, out: Optional[str] = None, extra: Optional[List[str]] = None,
                verbose: bool = False) -> str:
    headers = [os.path.join(INCLUDE, h) for h in ("r2l.h", "r2l_mixer.h")]
    return _compile(os.path.join(MIXER_CSRC, "mixer.cu"), out or MIXER_LIB, mixer_sources() + headers, force, extra, verbose)


def build(force: bool = False, out: Optional[str] = None, extra: Optional[List[str]] = None, verbose: bool = False) -> str:
    """Builds libr2l.so (or only that, at ``out``) and libr2l_mixer.so; returns the path of the first."""
    lib = _compile(os.path.join(CSRC, "r2l.cu"), out or LIB, sources() + [os.path.join(INCLUDE, "r2l.h")], force, extra, verbose)
    if out is None:
        build_mixer(force, None, extra, verbose)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
