"""Build the gfx950 HIP libraries in-tree: indexer_topk_long_amd/_lib/liblitetopk.so (the
fused Indexer-TopK, the paged cache's operators and those of prompts), ltk_bind.so (the
Python entry of the latter two) and indexer_topk_long_amd/_lib/libltkpeak.so (the achievable-peak
microbenchmarks the benchmark reports beside the vendor peaks).

    python -m indexer_topk_long_amd.build [-v]
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_NAME = "liblitetopk.so"
PEAK_SRC = os.path.join(PKG, "peak", "peak.hip")
PEAK_LIB = "libltkpeak.so"
BIND_SRCS = [os.path.join(CSRC, n) for n in ("attend_bind.cpp", "prompt_bind.cpp")]
BIND_LIB = "ltk_bind.so"
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
    # packed fp32 VALU forms stay off: scalar fp32 only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def lib_path() -> str:
    return os.path.join(OUT_DIR, LIB_NAME)


def bind_path() -> str:
    return os.path.join(OUT_DIR, BIND_LIB)


def _compile_bind(src: str, verbose: bool) -> str:
    """The compiled Python entries: host code against torch's headers."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", "/opt/rocm/include", "-isystem",
           sysconfig.get_paths()["include"], "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}{r.stderr}")
    return obj


def peak_lib_path() -> str:
    return os.path.join(OUT_DIR, PEAK_LIB)


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "is not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msg}")
    if verbose and msg.strip():
        print(msg)
    return obj


def build(verbose: bool = False) -> str:
    """Compile every HIP source for gfx950 and link the shared library. Returns its path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 3, 8)) as ex:
        binds = [ex.submit(_compile_bind, src, verbose) for src in BIND_SRCS]
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs + [PEAK_SRC]))
        bind_objs = [b.result() for b in binds]
    peak_obj = objs.pop()
    for out, inputs in ((lib_path(), objs), (peak_lib_path(), [peak_obj])):
        tmp = out + ".tmp"
        cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *inputs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
        os.replace(tmp, out)
    tmp = bind_path() + ".tmp"
    import torch   # its libraries are in the process before this one is loaded: no path to them is kept
    r = subprocess.run(["g++", "-shared", "-o", tmp, *bind_objs, "-L", OUT_DIR, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN", "-L",
                        os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
                        "-lc10_hip"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, bind_path())
    return lib_path()


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
