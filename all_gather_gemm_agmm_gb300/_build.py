"""Build the sm_103a shared library ``libagmm.so`` in-tree with nvcc.

The translation units (kernel variants in three groups, selection and launch,
C ABI, allocation-free entry point; the attention and the feed-forward operators'
kernels and C ABI)
compile in parallel to objects under
``_build/`` and link, with the CUDA runtime linked statically, into
``all_gather_gemm_agmm_gb300/libagmm.so``.  No cmake, one ``-gencode``.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
CSRC_ATTENTION = os.path.join(PKG, "csrc_attention")
CSRC_FEEDFORWARD = os.path.join(PKG, "csrc_feedforward")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libagmm.so")
SOURCES = ["agmm_select_rows_a1.cu", "agmm_select_rows_a2.cu", "agmm_select_swap.cu", "agmm_kernels.cu",
           "agmm_api.cpp", "agmm_noalloc.cu"]
ATTENTION_SOURCES = ["norm_rope.cu", "attn_prompt.cu", "attn_tree.cu", "attn_launch.cu", "attn_api.cpp"]
FEEDFORWARD_SOURCES = ["ff_wide_plain.cu", "ff_wide_gated.cu", "ff_wide_linear.cu", "ff_narrow_plain.cu",
                       "ff_narrow_gated.cu", "ff_narrow_linear.cu", "ff_swap_plain.cu", "ff_swap_gated.cu",
                       "ff_swap_linear.cu", "ff_wide_two.cu", "ff_narrow_two.cu", "ff_launch.cu", "ff_pointwise.cu", "layer_norm.cu", "ff_api.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libagmm.so")
    return cand


def _deps():
    files = [os.path.join(d, f) for d in (CSRC, CSRC_ATTENTION, CSRC_FEEDFORWARD, INCLUDE) for f in os.listdir(d)]
    files.append(os.path.abspath(__file__))
    return files


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _deps())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC, "-I", CSRC_ATTENTION, "-I", CSRC_FEEDFORWARD]
    if ptxas_info:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc] + common + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if ptxas_info or verbose:
            sys.stderr.write(r.stderr)
        return obj

    sources = [os.path.join(CSRC, f) for f in SOURCES] + [os.path.join(CSRC_ATTENTION, f) for f in ATTENTION_SOURCES]
    sources += [os.path.join(CSRC_FEEDFORWARD, f) for f in FEEDFORWARD_SOURCES]
    with ThreadPoolExecutor(max_workers=len(sources)) as ex:
        objs = list(ex.map(compile_one, sources))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "--cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
