"""Builds libfckl.so in-tree with nvcc for sm_100a (no GPU needed)."""
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfckl.so")
SOURCES = ["fckl.cu", "ce.cu", "norm.cu"]
HEADERS = ["ptx.cuh", "vec.cuh", "reduce.cuh", "gemm.cuh", "epilogues.cuh", "rows.cuh", "ce.cuh",
           "norm.cuh", "host.cuh"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def needs_rebuild() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "fckl.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, verbose) -> bool:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
    elif verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr)
    return r.returncode == 0


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not needs_rebuild():
        return LIB
    flags = ["-O3", "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo",
             "-Xcompiler", "-fPIC,-O3", "-I", INCLUDE, "-I", CSRC] + list(extra)
    with tempfile.TemporaryDirectory() as tmp:
        objs = [os.path.join(tmp, f + ".o") for f in SOURCES]
        cmds = [[nvcc_path()] + flags + ["-c", os.path.join(CSRC, f), "-o", o]
                for f, o in zip(SOURCES, objs)]
        with ThreadPoolExecutor() as pool:  # one nvcc per translation unit
            done = list(pool.map(lambda c: _run(c, verbose), cmds))
        if all(done):
            done.append(_run([nvcc_path(), "-shared", "-gencode", "arch=compute_100a,code=sm_100a",
                              "-o", LIB + ".tmp"] + objs, verbose))
    if not all(done):
        raise RuntimeError("nvcc failed building libfckl.so")
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [])
