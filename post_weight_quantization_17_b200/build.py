"""Builds libgptq_b200.so in-tree from csrc/*.cu for sm_100a with nvcc.

Usage: python post_weight_quantization_17_b200/build.py [--force] [--verbose-ptxas]
(run by path: importing the package would load the library it builds)
The library is rebuilt only when a source file, the public header or the flags change.
"""
from __future__ import annotations

import concurrent.futures
import glob
import hashlib
import os
import re
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgptq_b200.so")
BUILD_DIR = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
# Kernels whose roles hand registers to one another (setmaxnreg): a launch has to bring this many a thread, or
# a role would wait for registers that the block does not own.
LAUNCH_REGISTERS = {"k_lora_tc": 96}
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + os.path.join(ROOT, "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _digest(extra: list[str]) -> str:
    h = hashlib.sha256()
    files = _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(ROOT, "include", "gptq.h")]
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH + FLAGS + extra).encode())
    return h.hexdigest()


def check_registers(log: str) -> int:
    """ptxas -v output: raises if a kernel of LAUNCH_REGISTERS got fewer registers; how many it found."""
    found, name = 0, None
    for line in log.splitlines():
        entry = re.search(r"Compiling entry function '(\w+)'", line)
        used = re.search(r"Used (\d+) registers", line)
        if entry:
            name = next((k for k in LAUNCH_REGISTERS if f"{len(k)}{k}I" in entry.group(1)), None)
        elif used and name:
            if int(used.group(1)) < LAUNCH_REGISTERS[name]:
                raise RuntimeError(f"{name} was compiled with {used.group(1)} registers, it needs "
                                   f"{LAUNCH_REGISTERS[name]}")
            found, name = found + 1, None
    return found


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    digest = _digest(extra)
    stamp = LIB + ".sha256"
    if not force and os.path.exists(LIB) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == digest:
                return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        counted = os.path.splitext(os.path.basename(src))[0] in LAUNCH_REGISTERS
        cmd = [NVCC, *ARCH, *FLAGS, *(["-Xptxas", "-v"] if counted else extra), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        if counted and not check_registers(r.stderr):
            raise RuntimeError(f"no register counts for {src}:\n{r.stderr}")
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        results = list(ex.map(compile_one, _sources()))
    if ptxas_verbose:
        for _, err in results:
            sys.stderr.write(err)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart", "-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(digest)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_verbose="--verbose-ptxas" in sys.argv))
