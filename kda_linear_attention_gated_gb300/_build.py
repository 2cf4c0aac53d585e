"""In-tree build of the two CUDA libraries (sm_103a only).

    libkda_h0.so  fp32 state pool   (-DKDA_STATE16=0)
    libkda_h1.so  fp16 state pool   (-DKDA_STATE16=1)

Both come from the same source files; the pool dtype is a compile-time
constant, as the _h0/_h1 kernel names of ROCm/ATOM pull request 2945 (Changes)
make it.  The libraries link the shared CUDA runtime, so they share the
runtime instance (and the streams) of the PyTorch process that loads them.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
LIB_DIR = os.path.join(PKG_DIR, "lib")
SOURCES = [os.path.join(CSRC, f) for f in ("kda_api.cu", "kda_common.cuh", "kda_decode_tma.cuh",
                                          "kda_verify_tma.cuh", "kda_conv.cuh", "kda_ckpt.cuh",
                                          "kda_prefill_chunk.cuh", "kda_stage.cuh", "kda_host.cuh",
                                          "kda_layer_api.cu", "kda_kv4.cuh", "kda_kv4_tree.cuh", "kda_norm.cuh",
                                          "kda_tree_api.cu", "kda_tree.cuh", "kda_accept.cuh")] + [os.path.join(INCLUDE, "kda.h")]

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def lib_path(state16: bool) -> str:
    return os.path.join(LIB_DIR, f"libkda_h{int(bool(state16))}.so")


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KDA CUDA libraries cannot be built")


def _stale(out: str) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(s) > t for s in SOURCES)


UNITS = [os.path.join(CSRC, f) for f in ("kda_api.cu", "kda_layer_api.cu", "kda_tree_api.cu")]


def _flags(state16: bool) -> list[str]:
    return [_nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17",
            "-Xcompiler", "-fPIC", "-cudart", "shared",
            f"-I{INCLUDE}", f"-DKDA_STATE16={int(bool(state16))}"]


def nvcc_command(state16: bool, out: str, extra: list[str] | None = None) -> list[str]:
    """One command that builds a whole library (build() compiles its units at the same time)."""
    return [*_flags(state16), "-shared", *(extra or []), *UNITS, "-o", out]


def _run(what: str, cmd: list[str]) -> None:
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        raise RuntimeError(f"nvcc failed for {what}:\n{proc.stderr}")


def build(force: bool = False) -> list[str]:
    """Compile both libraries, their units in parallel, if any source is newer than them."""
    stale = [s for s in (False, True) if force or _stale(lib_path(s))]
    if stale:
        os.makedirs(LIB_DIR, exist_ok=True)
        with tempfile.TemporaryDirectory(dir=LIB_DIR) as tmp:
            def unit(job):
                state16, src = job
                obj = os.path.join(tmp, f"{os.path.basename(src)[:-3]}_h{int(state16)}.o")
                _run(os.path.basename(src), [*_flags(state16), "-c", src, "-o", obj])
                return state16, obj
            jobs = [(s, u) for u in UNITS for s in stale]
            with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
                objects = list(ex.map(unit, jobs))
            for s in stale:
                out = os.path.join(tmp, os.path.basename(lib_path(s)))
                _run(os.path.basename(out), [*_flags(s), "-shared", *(o for t, o in objects if t == s), "-o", out])
                os.replace(out, lib_path(s))
    return [lib_path(s) for s in (False, True)]


if __name__ == "__main__":
    for p in build(force=True):
        print(p)
