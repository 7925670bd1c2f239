"""Build libpi.so (the HIP kernels and the C ABI) in-tree for gfx950.

    python -m activation_sparse_rank_amd.build [--jobs N]

Every HIP source under csrc/ is compiled with hipcc for gfx950 only and linked
into ``activation_sparse_rank_amd/libpi.so``.  Objects go to ``_build/`` at
the repository root.  ``bind_attn.cpp`` (host code: the attention side's checks
of tensors) becomes the Python module ``_attn.so`` beside it.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpi.so")
BIND = os.path.join(PKG, "_attn.so")

SOURCES = ["abi.hip", "k_predict.hip", "k_compact.hip", "k_gather.hip", "k_mfma.hip", "k_q4.hip", "k_place.hip", "k_stream.hip",
           "abi_attn.hip", "k_rope.hip", "k_kvcache.hip", "k_attend.hip", "k_evict.hip"]

ARCH = "gfx950"
CFLAGS = [
    "-x", "hip", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-function",
    # Packed fp32 VALU instructions stay off in every HIP object.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc(), *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _bind() -> str:
    """Compile the Python module _attn against the installed torch."""
    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    tmp = BIND + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"]]
    for d in (*include_paths(), os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include")):
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "bind_attn.cpp"), "-o", tmp]
    for d in library_paths():
        cmd += ["-L", d]
    cmd += ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_hip", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for bind_attn.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    return BIND


def build(jobs: int | None = None, verbose: bool = False) -> str:
    """Compile every source and link libpi.so; returns the library path."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(8, len(SOURCES))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        bind = ex.submit(_bind)
        objs = list(ex.map(_compile, SOURCES))
        bind.result()
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB} and {BIND}")
    return LIB


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--jobs", type=int, default=None)
    args = ap.parse_args(argv)
    build(args.jobs, verbose=True)
    return 0


if __name__ == "__main__":
    sys.exit(main())
