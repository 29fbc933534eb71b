"""Build libe2f.so (all CUDA sources, sm_100a) in-tree.

    python -m atomistic_mlip_b200.build [--force]

Objects go to ``_build/`` at the repository root; the shared library is
written next to this file, where the binding loads it.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "libe2f.so")
BUILD_DIR = os.path.join(ROOT, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "-I", os.path.join(ROOT, "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(p) <= t for p in _deps())


# Kernels that redistribute their registers (setmaxnreg), by mangled name, and the
# registers a thread that they must be launched with to do so.
REDISTRIBUTED = [(re.compile(r"gemm_reg_kernelI"), 72),
                 (re.compile(r"gemm_tma_kernelILb[01]ELb[01]ELi\d+ELb1E"), 168)]   # LONGK


def check_registers(ptxas_report: str) -> int:
    """Number of such kernels in ptxas's report; RuntimeError if one was compiled to
    fewer registers than it hands out (it would wait for ever)."""
    name, seen = "", 0
    for line in ptxas_report.splitlines():
        m = re.search(r"Compiling entry function '([^']+)'", line)
        if m:
            name = m.group(1)
        m = re.search(r"Used (\d+) registers", line)
        if not m:
            continue
        for pattern, regs in REDISTRIBUTED:
            if pattern.search(name):
                seen += 1
                if (int(m.group(1)) + 7) // 8 * 8 < regs:
                    raise RuntimeError(f"{name} was compiled to {m.group(1)} registers, it hands out {regs}")
        name = ""
    return seen


def _compile(src: str, extra, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-Xptxas", "-v", "-c", src, "-o", obj]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if verbose or r.returncode or "warning" in r.stdout:
        sys.stderr.write(r.stdout)
    r.check_returncode()
    check_registers(r.stdout)
    return obj


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return OUT
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra, verbose), _sources()))
    tmp = OUT + ".tmp"
    subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcublas"])
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
