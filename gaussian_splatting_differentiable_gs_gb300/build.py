"""Builds libgs103.so (the CUDA library behind include/gs.h) in-tree.

Each .cu file under csrc/ is compiled for sm_103a in parallel, then linked
into gaussian_splatting_differentiable_gs_gb300/libgs103.so.  Objects go to
gaussian_splatting_differentiable_gs_gb300/_build/ (git-ignored).
"""
import concurrent.futures as cf
import glob
import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgs103.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def _nvcc():
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def _check_registers(src, log):
    """A kernel whose warps share out the registers of its launch states their number
    (kLaunchRegs, in the file of <file>_kernel); the library refuses to launch it with
    any other.  Raises here if the compiler gave another number."""
    want = re.search(r"kLaunchRegs = (\d+)", open(src).read())
    if not want:
        return
    kernel = os.path.basename(src)[:-3] + "_kernel"
    used = [int(n) for n in re.findall(
        r"Compiling entry function '\w*?\d%s\w*'(?:(?!Compiling)[\s\S])*?Used (\d+) registers" % kernel, log)]
    if not used or set(used) != {int(want.group(1))}:
        raise RuntimeError("%s: %s was given %s registers a thread, its launch needs %s"
                           % (src, kernel, sorted(set(used)) or "no known number of", want.group(1)))


def _compile(src, verbose):
    obj = os.path.join(OUT, os.path.basename(src) + ".o")
    cmd = [_nvcc()] + ARCH + FLAGS + ["-Xptxas", "-v", "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    _check_registers(src, r.stderr)
    return obj, r.stderr


def build(force=False, verbose=False):
    if (not force and os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(p) for p in _deps())):
        return LIB
    os.makedirs(OUT, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cmd = [_nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
