"""Build libbq.so (the sm_100a kernels behind include/bq.h) in-tree with nvcc.

Each .cu under csrc/ is compiled to an object in parallel, then linked into a
shared library next to this file.  The CUDA runtime is linked statically, so
the library only needs the NVIDIA driver at run time.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import re
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libbq.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "--expt-relaxed-constexpr", "-Xcompiler", "-Wall"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libbq.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


# Kernels whose warps share out (setmaxnreg) the registers that a CTA is launched with: more than that and they wait for
# ever, so each variant has to be compiled to the very count that the source's constant names.  kernel, constant by file
EXACT_REGISTERS = {"kv4_prefill.cu": ("kv4_prefill_kernel", "kLaunchRegs")}


def registers_of(ptxas: str, kernel: str) -> dict:
    """{variant: registers} of a kernel, from what `ptxas -v` printed."""
    found, name = {}, None
    for line in ptxas.splitlines():
        m = re.search(r"Compiling entry function '(\w+)'", line)
        name = m.group(1) if m else name
        m = re.search(r"Used (\d+) registers", line)
        if m and name and kernel in name:
            found[name] = int(m.group(1))
    return found


def check_registers(src: str, text: str, ptxas: str) -> None:
    """Fails the build where a kernel of EXACT_REGISTERS was not compiled to its source's count."""
    kernel, constant = EXACT_REGISTERS[os.path.basename(src)]
    want = int(re.search(constant + r" = (\d+)", text).group(1))
    found = registers_of(ptxas, kernel)
    wrong = {k: v for k, v in found.items() if v != want}
    if wrong or not found:
        raise RuntimeError(f"{src}: {kernel} needs {want} registers in every variant ({constant} and the shares of its "
                           f"roles), the compiler gave {wrong or 'no figures'}")


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    exact = os.path.basename(src) in EXACT_REGISTERS
    if exact and not extra:
        extra = ["-Xptxas", "-v"]
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if exact:
        with open(src) as f:
            check_registers(src, f.read(), r.stderr)
    if r.stderr.strip() and "ptxas info" in r.stderr:
        with open(obj + ".ptxas.txt", "w") as f:
            f.write(r.stderr)
    return obj


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile libbq.so if it is missing or older than its sources; return its path."""
    if not force and not stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra), _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, ptxas_verbose="-v" in sys.argv))
