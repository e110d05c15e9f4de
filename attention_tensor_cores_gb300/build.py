"""Builds libfmha.so in place from csrc/*.cu with nvcc for sm_103a only, and the Python binding of its
paged-cache entry points, _binding.so, from csrc/binding.cpp with g++ against the installed torch.

Each translation unit is compiled in parallel (nvcc -c), then linked into one shared library.
Objects go to attention_tensor_cores_gb300/_build/ (git-ignored).  Re-running only recompiles
what changed (source or any header newer than its object).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfmha.so")
BINDING = os.path.join(PKG, "_binding.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    p = os.path.join(home, "bin", "nvcc")
    return p if os.path.exists(p) else "nvcc"


def _headers() -> list[str]:
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(ROOT, "include", "fmha.h")]


# Per-file register ceilings: the row-tile kernel runs 10 warps per SM, so up to 200 registers per
# thread fit, and the softmax keeps a 128-column row of S in registers.
PER_FILE_FLAGS = {}


def _compile(src: str, obj: str, extra: list[str]) -> tuple[str, str]:
    cmd = [_nvcc()] + ARCH + NVCC_FLAGS + PER_FILE_FLAGS.get(os.path.basename(src), []) + extra + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return src, r.stdout + r.stderr


def _build_binding(force: bool) -> None:
    """_binding.so, which fits one torch and one Python: remade when either or its sources changed."""
    src, header = os.path.join(CSRC, "binding.cpp"), os.path.join(ROOT, "include", "fmha.h")
    made_for = f"torch {importlib.metadata.version('torch')}, python {sys.version}"
    note = os.path.join(BUILD, "binding.txt")
    if not force and os.path.exists(BINDING) and os.path.exists(note) and open(note).read() == made_for and \
            os.path.getmtime(BINDING) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    tmp = BINDING + f".tmp{os.getpid()}"
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", src, "-o", tmp] + [f"-I{d}" for d in inc] + \
        ["-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(note, "w") as f:
        f.write(made_for)


def build(force: bool = False, verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile every csrc/*.cu and link libfmha.so; returns the library path."""
    extra = list(extra or [])
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = max(os.path.getmtime(h) for h in _headers())
    jobs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or extra or not os.path.exists(o) or os.path.getmtime(o) < max(os.path.getmtime(s), hdr_time):
            jobs.append((s, o))
    with cf.ThreadPoolExecutor(max_workers=min(len(jobs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_build_binding, force)
        if jobs:
            for src, log in ex.map(lambda j: _compile(j[0], j[1], extra), jobs):
                if verbose and log.strip():
                    print(f"--- {os.path.basename(src)}\n{log}", file=sys.stderr)
        binding.result()
    if jobs or not os.path.exists(LIB):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [_nvcc()] + ARCH + ["-shared", "-o", tmp] + objs + ["-lcudart_static", "-ldl", "-lrt", "-lpthread"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    ptxas = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(force="--force" in sys.argv or bool(ptxas), verbose=v or bool(ptxas), extra=ptxas))
