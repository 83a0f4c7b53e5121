"""Build libbsfa.so in-tree for sm_103a with nvcc (no cmake, no torch), and the
torch binding of the 16-bit cache with the host compiler.

    python -m block_sparse_gated_gb300.build [--force] [--jobs N]

Translation units are compiled in parallel; the shared libraries land next to
this file, where the package loads them from.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libbsfa.so")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_STAMP = os.path.join(OBJDIR, "binding.torch")  # the torch that it was built with

SOURCES = ["bsfa_api.cu", "inst_fwd_d128.cu", "inst_fwd_d64.cu", "inst_fwd_vall.cu",
           "inst_calib.cu", "inst_fwd_paged_d128.cu", "inst_fwd_paged_d64.cu", "inst_fwd_corr.cu",
           "bsfa_noalloc.cu", "inst_xs.cu", "inst_xs224.cu", "bsfa_cache4.cu", "bsfa_decode4.cu",
           "bsfa_cache16.cu", "bsfa_decode16.cu", "inst_decode16_d64_bf16.cu",
           "inst_decode16_d64_f16.cu", "inst_decode16_d128_bf16.cu", "inst_decode16_d128_f16.cu",
           "inst_decode16_wide_d64.cu", "inst_decode16_wide_d128.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _deps_mtime() -> float:
    t = 0.0
    for d in (CSRC, INCLUDE):
        for f in os.listdir(d):
            t = max(t, os.path.getmtime(os.path.join(d, f)))
    return t


def _compile(src: str, verbose_ptxas: bool) -> tuple[str, str]:
    obj = os.path.join(OBJDIR, src.replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src),
           "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    with open(obj + ".log", "w") as f:  # what the compiler had to say, spills among it
        f.write(r.stdout + r.stderr)
    return obj, r.stdout + r.stderr


def _torch_place() -> tuple[str, str] | None:
    """Where torch lies and its version, without importing it; None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    root = os.path.dirname(spec.origin)
    with open(os.path.join(root, "version.py")) as f:
        return root, re.search(r"__version__ = '([^']*)'", f.read()).group(1)


def _build_binding(root: str, version: str) -> None:
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = BINDING + ".tmp"
    inc = [INCLUDE, os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           *[x for i in inc for x in ("-isystem", i)], os.path.join(CSRC, "binding.cpp"),
           "-o", tmp, "-L", PKG, "-l:libbsfa.so", "-L", os.path.join(root, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(version)


def _binding_is_current(version: str) -> bool:
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) < _deps_mtime() or \
            not os.path.exists(BINDING_STAMP):
        return False
    with open(BINDING_STAMP) as f:
        return f.read() == version


def build(force: bool = False, jobs: int | None = None, verbose_ptxas: bool = False) -> str:
    """Compile every translation unit, link libbsfa.so and build the torch
    binding; returns the library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < _deps_mtime():
        _build_library(jobs, verbose_ptxas)
    place = _torch_place()  # the library itself does not need it
    if place is not None and (force or not _binding_is_current(place[1])):
        _build_binding(*place)
    return LIB


def _build_library(jobs: int | None, verbose_ptxas: bool) -> None:
    jobs = jobs or min(len(SOURCES), os.cpu_count() or 1)
    with cf.ThreadPoolExecutor(jobs) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), SOURCES))
    if verbose_ptxas:
        for _, log in results:
            sys.stdout.write(log)
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--jobs", type=int, default=None)
    ap.add_argument("--ptxas-v", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, jobs=a.jobs, verbose_ptxas=a.ptxas_v))
