"""Build step for the CUDA library: compiles csrc/*.cu for sm_100a with nvcc and
links libatf.so next to this file (in-tree, so it ships with the package), and
csrc/tensor_calls.cpp, its calls on torch tensors, to a module named after the
torch and Python that it was built against."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libatf.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _headers():
    return glob.glob(os.path.join(SRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    if _stale(obj, [src] + _headers()):
        cmd = [NVCC, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
    return obj


def tensor_calls_path() -> str:
    """The module for this torch and this Python, whose C++ and C interfaces it is compiled against: after an
    upgrade of either it is another file, to be built anew."""
    import torch

    return os.path.join(HERE, f"_tensor_calls-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _build_tensor_calls(force):
    src = os.path.join(SRC, "tensor_calls.cpp")
    try:
        import torch

        target = tensor_calls_path()
    except ImportError:
        print("torch is not installed: its module is left out, the C library is complete", file=sys.stderr)
        return
    if not force and not _stale(target, [src, os.path.join(ROOT, "include", "atf.h")]):
        return

    home = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(NVCC) or NVCC)))  # NVCC may be a bare name
    inc = [sysconfig.get_paths()["include"], os.path.join(home, "include"),
           os.path.join(home, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    tmp = target + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *("-I" + d for d in inc), src, "-o", tmp,
           "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, target)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(SRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        calls = ex.submit(_build_tensor_calls, force)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        if force or _stale(LIB, objs):
            tmp = LIB + f".tmp{os.getpid()}"
            cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        calls.result()  # the C library does not wait for torch's headers, or fail with them
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
