"""Builds libmuon_ns.so in-tree with nvcc for sm_103a (no CMake, no torch extension).

The translation units compile in parallel; the shared library links the CUDA
runtime statically so it loads on a host without a GPU driver (only the
host-side entry points work there).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libmuon_ns.so")
SOURCES = ["engine.cu", "tc_gemm.cu", "simt_gemm.cu", "elementwise.cu", "adamw.cu", "planner.cpp",
           "train_abi.cu", "clip.cu", "rms_norm.cu", "fp8_quant.cu", "fp8_gemm.cu",
           "fp8_few.cu", "block_abi.cu", "block_norm.cu", "block_norm_grad.cu", "gated.cu", "fp8_transpose.cu"]
# (source, object, defines): compiled once for each type and alignment, in parallel
ROWS = [(src, f"{src[:-3]}_{name}{'_any' if anywhere else ''}",
         [f"-DMUON_ROWS_T={t}", f"-DMUON_ROWS_ANYWHERE={'true' if anywhere else 'false'}"])
        for src in ("block_norm_rows.cu", "block_norm_grad_rows.cu")
        for name, t in (("bf16", "__nv_bfloat16"), ("fp16", "__half"), ("fp32", "float"))
        for anywhere in (False, True)]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                   f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", *extra]


def _stale(lib, deps):
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose=False, force=False, extra=()) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "muon_ns.h")]
    if not force and not _stale(LIB, deps):
        return LIB
    cc = nvcc()
    objs = []

    def comp(unit):
        src, name, defines = unit
        obj = os.path.join(OUT_DIR, name + ".o")
        cmd = [cc, *_flags(extra), *defines, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stdout.write(r.stdout + r.stderr)
        return obj

    units = ROWS + [(src, os.path.splitext(src)[0], []) for src in SOURCES]  # the longest first
    with cf.ThreadPoolExecutor(max_workers=len(units)) as ex:
        objs = list(ex.map(comp, units))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if v else []
    print(build(verbose=v, force=True, extra=extra))
