"""Compile the CUDA library in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel, then linked into
``onnx_recurrent_gb300/_build/libonnx_recurrent_gb300.so`` (static cudart, no
torch types).  A stamp of the sources and flags skips up-to-date builds.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libonnx_recurrent_gb300.so")
SOURCES = ["rnn_api.cpp", "k_proj.cu", "k_proj_tc.cu", "k_misc.cu", "k_recur_rnn.cu", "k_recur_gru.cu",
           "k_recur_lstm.cu", "k_recur_tc.cu", "k_cell.cu", "rnn_static.cu", "k_wave_rnn.cu", "k_wave_gru.cu",
           "k_wave_lstm.cu", "k_clus_rnn.cu", "k_clus_gru.cu", "k_clus_lstm.cu", "ssm_api.cpp", "k_ssm_conv.cu", "k_ssm_scan.cu",
           "k_ssm_scan_grad.cu", "k_ssm_step.cu", "k_scores.cu"]
HEADERS = ["rnn_internal.h", "exact_math.cuh", "io_types.cuh", "tma.cuh", "k_recur.cuh", "k_recur2.cuh",
           "k_wave.cuh", "ssm_internal.h", "ssm_math.cuh", "ssm_tile.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return cand


def _stamp(extra_flags) -> str:
    h = hashlib.sha256()
    for name in SOURCES + HEADERS:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(ROOT, "include", "onnx_recurrent.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(FLAGS + list(extra_flags)).encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build the shared library if needed and return its path."""
    os.makedirs(BUILD, exist_ok=True)
    stamp_path = os.path.join(BUILD, "stamp")
    stamp = _stamp(extra_flags)
    if not force and os.path.exists(LIB) and os.path.exists(stamp_path):
        with open(stamp_path) as f:
            if f.read().strip() == stamp:
                return LIB
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB + f".{os.getpid()}.tmp"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp_path, "w") as f:
        f.write(stamp)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
