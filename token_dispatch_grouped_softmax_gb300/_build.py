"""In-tree build of libmoe_gb300.so for sm_103a (nvcc, no cmake).

Each .cu file is compiled in parallel into _build/, then linked into a shared
library next to this file.  The CUDA runtime is linked as a shared library so
the process shares one runtime (current device, streams) with PyTorch.  Beside
it the Python extension of the calls of a decode step is built from
csrc/binding.cpp with the host compiler, against Python's and torch's headers;
its file's name holds both versions, so that another torch or Python builds
its own.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_gb300.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def binding_path() -> str:
    """The extension's file, of this Python and this torch."""
    import torch

    return os.path.join(PKG, "_binding-%s%s" % (torch.__version__, sysconfig.get_config_var("EXT_SUFFIX")))


def up_to_date() -> bool:
    for out, deps in ((LIB, _deps()), (binding_path(), [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h")))):
        if not os.path.exists(out):
            return False
        t = os.path.getmtime(out)
        if not all(os.path.getmtime(d) <= t for d in deps):
            return False
    return True


def _build_binding(verbose):
    import torch

    root = os.path.dirname(os.path.abspath(torch.__file__))
    out = binding_path()
    tmp = out + ".%d.tmp" % os.getpid()
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi()),
           "-I" + os.path.join(root, "include"), "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           "-I" + sysconfig.get_paths()["include"], BINDING_SRC, "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed on %s:\n%s\n%s" % (cmd[0], BINDING_SRC, r.stdout, r.stderr))
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr)
    os.replace(tmp, out)


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """Compile and link libmoe_gb300.so and the extension when missing or older than their sources."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + ARCH + NVCC_FLAGS + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_build_binding, verbose)
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".%d.tmp" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs + \
        ["-Xlinker", "-rpath=/usr/local/cuda/lib64"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    binding.result()   # the library needs no torch: it is there even where the extension failed
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
