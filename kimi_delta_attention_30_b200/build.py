"""Build ``libkda.so`` (the C-ABI CUDA library) in-tree for sm_100a, and
``_torch_binding.so`` (torch tensors into the C ABI, host code) beside it.

Usage: ``python -m kimi_delta_attention_30_b200.build [--force]``.
Each ``csrc/*.cu`` is compiled by nvcc to an object under ``_build/`` (in
parallel), then linked into ``kimi_delta_attention_30_b200/libkda.so``.
Set ``KDA_NVCC_FLAGS`` to append flags (e.g. ``-Xptxas -v``).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import shlex
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libkda.so")
BINDING_SRC = os.path.join(CSRC, "torch_binding.cpp")
BINDING = os.path.join(PKG, "_torch_binding.so")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    return "nvcc"


def cuda_lib_dir() -> str:
    return os.path.join(os.path.dirname(os.path.dirname(nvcc())), "lib64")


FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _binding_target() -> str:
    """The torch and Python whose binary interfaces the binding is compiled to."""
    import torch
    return f"torch {torch.__version__} {torch.version.git_version}, {sys.implementation.cache_tag}"


def binding_built_for() -> str:
    """The same of the binding that is there, which carries it as text (read before it is loaded)."""
    try:
        with open(BINDING, "rb") as f:
            m = re.search(rb"kda binding built for \[([^\]]*)\]", f.read())
    except OSError:
        return "nothing"
    return m.group(1).decode() if m else "unknown"


def _binding_stale() -> bool:
    if not os.path.exists(BINDING) or binding_built_for() != _binding_target():
        return True
    t = os.path.getmtime(BINDING)
    return any(os.path.getmtime(p) > t for p in [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))


def build_binding(force: bool = False) -> str:
    """Compile the torch binding with g++ (links ``libkda.so`` beside it)."""
    if not force and not _binding_stale():
        return BINDING
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(cuda_lib_dir())
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f'-DKDA_BUILT_FOR="{_binding_target()}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
           *(f"-isystem{p}" for p in ext.include_paths()), BINDING_SRC, "-o", tmp, "-L", PKG, "-l:libkda.so", "-L", libs, "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        build_binding()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = shlex.split(os.environ.get("KDA_NVCC_FLAGS", ""))
    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs,
           "-L", cuda_lib_dir(), "-lcudart", "-Xlinker", "--no-undefined"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_binding(force)
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
