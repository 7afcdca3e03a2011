"""Build libbsa.so in-tree with nvcc for sm_100a.

    python -m block_sparse_attention_47_b200.build [--verbose]

Each .cu file under csrc/ is compiled in parallel to an object file under
_build/, then linked into block_sparse_attention_47_b200/libbsa.so (static
CUDA runtime, no other dependency).  Rebuilds only when a source or header
is newer than the library.
"""
import concurrent.futures as cf
import glob
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build", "bsa")
LIB = os.path.join(PKG, "libbsa.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]

# Kernels whose warps exchange registers: their split adds up to the threads
# times this many, and with any other number the exchange would not end
REGISTERS = {"packed_fwd_kernel": 168}


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(ROOT, "include", "*.h")) + [__file__])


def up_to_date():
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def check_registers(log, required=None):
    """Raises unless every kernel named in `required` is in ptxas' report with
    that many registers a thread."""
    required = REGISTERS if required is None else required
    used = re.findall(r"Compiling entry function '(\w+)'.*?Used (\d+) registers", log, re.S)
    for kernel, n in required.items():
        got = [int(r) for name, r in used if kernel in name]
        if not got or any(r != n for r in got):
            raise RuntimeError("%s has to take %d registers a thread; the compiler's report has %s"
                               % (kernel, n, sorted(set(got)) or "none"))


def build(verbose=False, force=False, ptxas_verbose=False):
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    def one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, "-Xptxas", "-v", "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(one, _sources()))
    failed = False
    for src, _, r in results:
        if verbose or r.returncode or ptxas_verbose:
            sys.stderr.write(r.stdout + r.stderr)
        if r.returncode:
            sys.stderr.write("nvcc failed on %s\n" % src)
            failed = True
    if failed:
        raise RuntimeError("libbsa.so build failed")
    check_registers("\n".join(r.stdout + r.stderr for _, _, r in results))
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp] + [obj for _, obj, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("libbsa.so link failed")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose="--verbose" in sys.argv, force=True, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB)
