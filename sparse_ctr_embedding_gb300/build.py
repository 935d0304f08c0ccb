"""Build the sm_103a shared library in-tree: sparse_ctr_embedding_gb300/_build/libemb_gb300.so.

nvcc compiles each translation unit that changed, in parallel, and links a shared library
with the CUDA runtime linked statically, exporting only the C ABI declared in
include/emb_gb300.h.
"""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD, "libemb_gb300.so")
HEADER = os.path.join(ROOT, "include", "emb_gb300.h")
SOURCES = ["emb_table.cu", "emb_fwd.cu", "emb_bwd.cu", "emb_pipe.cu", "emb_build.cu",
           "emb_fp8.cu", "emb_fp8_matmul.cu", "emb_norm_fwd.cu", "emb_norm_bwd.cu", "emb_adamw.cu",
           "emb_fp4.cu", "emb_fp4_matmul.cu", "emb_muon.cu", "emb_token.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC = os.environ.get("NVCC", "nvcc")
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
          "-I", os.path.join(ROOT, "include")]


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES] + [HEADER]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    common = max(os.path.getmtime(f) for f in [__file__, *_inputs()] if not f.endswith(".cu"))
    for src in SOURCES:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        newest = max(common, os.path.getmtime(os.path.join(CSRC, src)))
        if not force and os.path.exists(obj) and os.path.getmtime(obj) > newest:
            continue
        part = f"{obj}.tmp{os.getpid()}.o"      # an object that is there is whole
        cmd = [NVCC, *ARCH, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", part]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, obj, part, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, obj, part, p in procs:
        out, _ = p.communicate()
        if p.returncode == 0:
            os.replace(part, obj)
        else:
            failed.append(f"{src}:\n{out.decode(errors='replace')}")
        if p.returncode == 0 and verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
    if failed:
        raise RuntimeError("nvcc failed\n" + "\n".join(failed))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    subprocess.run([NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
