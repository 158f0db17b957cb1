"""Builds libecf8.so (host encoder + sm_100a decode kernels) in this directory."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SO = os.path.join(HERE, "libecf8.so")
# the same library with every kernel store and table read bounds-checked
# (-DECF8_CHECKED): a failed check sets ECF8_STATUS_BOUNDS instead of accessing
CHECKED_SO = os.path.join(HERE, "libecf8_checked.so")
SOURCES = [os.path.join(CSRC, f) for f in (
    "ecf8_host.cpp", "ecf8_decode.cu", "ecf8_pipeline.cpp", "ecf8_encode.cu", "ecf8_bf16_host.cpp", "ecf8_bf16_decode.cu",
    "ecf8_linear.cu", "ecf8_product_bf16.cu", "ecf8_product_bf16_back.cu", "ecf8_product_fp16.cu",
    "ecf8_product_fp16_back.cu", "ecf8_grad.cu")]
HEADERS = [os.path.join(ROOT, "include", "ecf8.h"),
           *(os.path.join(CSRC, f) for f in ("ecf8_format.h", "ecf8_tc.cuh", "ecf8_linear.cuh", "ecf8_product.cuh"))]
OBJECTS = os.path.join(HERE, "build")

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-Xfatbin", "-compress-all",
    "-Xcompiler", "-fPIC,-fopenmp,-O3",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def stale(so: str = SO) -> bool:
    if not os.path.exists(so):
        return True
    t = os.path.getmtime(so)
    return any(os.path.getmtime(f) > t for f in SOURCES + HEADERS)


def _run(cmd: list, out: str) -> None:
    """Runs a command that writes `out`: to a file of this process's own first, since others may build as well."""
    own = f"{out}.{os.getpid()}"
    subprocess.check_call([own if c == out else c for c in cmd])
    os.replace(own, out)


def _compile(source: str, checked: bool, force: bool, verbose: bool) -> str:
    """The object of one source.  The checked build has objects of its own where the checks make a difference."""
    with open(source) as f:
        checked = checked and "ECF8_CHECKED" in f.read()
    out = os.path.join(OBJECTS, os.path.basename(source) + (".checked.o" if checked else ".o"))
    if force or not os.path.exists(out) or any(os.path.getmtime(f) > os.path.getmtime(out) for f in [source, *HEADERS]):
        _run([nvcc(), *(["-Xptxas=-v"] if verbose else []), *NVCC_FLAGS, *(["-DECF8_CHECKED"] if checked else []),
              "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-c", "-o", out, source], out)
    return out


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    """Compiles what is out of date, the sources beside each other, and links."""
    so = CHECKED_SO if checked else SO
    if force or stale(so):
        os.makedirs(OBJECTS, exist_ok=True)
        with concurrent.futures.ThreadPoolExecutor(os.cpu_count() or 1) as pool:
            objects = list(pool.map(lambda f: _compile(f, checked, force, verbose), SOURCES))
        _run([nvcc(), *NVCC_FLAGS, "-shared", "-o", so, *objects, "-lgomp"], so)
    return so


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, checked="--checked" in sys.argv))
