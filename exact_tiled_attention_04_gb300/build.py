"""Build the sm_103a attention library in-tree with nvcc.

Each CUDA translation unit is compiled in its own nvcc process (in parallel)
for exactly one target, ``-gencode arch=compute_103a,code=sm_103a``, then
linked into ``libfa_gb300.so`` beside this file.  The CUDA runtime is linked
statically; the driver API is reached through the runtime's entry-point
query, so nothing else is linked.

    python -m exact_tiled_attention_04_gb300.build [--force] [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "libfa_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
SOURCES = ["fa_api.cu", "fa_fwd_bf16.cu", "fa_fwd_f16.cu", "fa_fwd_tf32.cu", "fa_merge.cu",
           "fa_bwd_api.cu", "fa_bwd_bf16.cu", "fa_bwd_f16.cu", "fa_bwd_aux.cu", "fa_pipeline.cu",
           "fa_dec_bf16.cu", "fa_dec_f16.cu", "fa_kv4_api.cu", "fa_kv4_store.cu", "fa_kv4_fwd.cu",
           "fa_kv4_evict.cu", "fa_weights.cu", "fa_packed_api.cu", "fa_packed_aux.cu", "fa_packed_bf16.cu",
           "fa_packed_f16.cu", "fa_paged_api.cu", "fa_paged_store.cu", "fa_paged_bf16.cu", "fa_paged_f16.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _deps() -> list[str]:
    out = [os.path.join(INCLUDE, "fa.h")]
    for name in os.listdir(CSRC):
        out.append(os.path.join(CSRC, name))
    return out


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose_ptxas: bool = False, extra: list[str] | None = None) -> str:
    """Compile and link; returns the library path."""
    if not force and not verbose_ptxas and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = [cc, "-std=c++17", "-O3", *ARCH, "-lineinfo", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        common += ["-Xptxas", "-v"]
    common += list(extra or [])

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = common + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    with ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose_ptxas:
        for _, log in results:
            sys.stdout.write(log)
    tmp = f"{LIB_PATH}.{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
