"""Builds the CUDA library libgdr.so (sm_103a) in-tree, next to this file.

Each translation unit is compiled by its own nvcc process (in parallel), then
linked into one shared library that exports the C ABI of include/gdr.h.
"""
import os
import re
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgdr.so")
SOURCES = ["gdr_api.cu", "gdr_prep_kda.cu", "gdr_prep_gdn.cu", "gdr_states_tc.cu", "gdr_main_kda.cu", "gdr_main_gdn.cu", "gdr_out.cu", "gdr_conv.cu",
           "gdr_block_api.cu", "gdr_glr_fwd.cu", "gdr_glr_bwd.cu", "gdr_norm.cu", "gdr_conv_fwd.cu",
           "gdr_dla_api.cu", "gdr_dla.cu", "gdr_dla_step.cu", "gdr_e4m3_api.cu", "gdr_linear.cu", "gdr_quant.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC = os.environ.get("NVCC", "nvcc")
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-Xptxas", "-v"]
# Kernels whose warps move registers among themselves (setmaxnreg): the shares have to come out of what the compiler
# gave a thread at the launch, or the warps that ask for more wait for ever.
REGISTERS = {"gdr_dla.cu": (r"k_dlaILi\d+ELi\d+E", 96), "gdr_linear.cu": (r"k_linearILb1ELi256E", 168)}


def check_registers(src, log):
    """Raises where the compiler's report (-Xptxas -v) gives a kernel of REGISTERS another number of registers."""
    if src not in REGISTERS:
        return
    kernel, want = REGISTERS[src]
    for name, got in re.findall(r"entry function '(\S+)' for .*?Used (\d+) registers", log, re.S):
        if re.search(kernel, name) and int(got) != want:
            raise RuntimeError("%s: the compiler gave %s %s registers a thread, and its warps' shares are made for %d"
                               % (src, name, got, want))


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(HERE, "..", "include", "gdr.h"))
    return files


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    deps = _deps()
    if not force and not _stale(LIB, deps + [os.path.abspath(__file__)]):
        return LIB
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [NVCC, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        check_registers(src, r.stdout + r.stderr)
        return obj, r.stderr

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results] + ["-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose="-v" in sys.argv))
