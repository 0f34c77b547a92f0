"""Build the CUDA library libfp8idx.so in-tree for sm_100a with nvcc."""
from __future__ import annotations

import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfp8idx.so")
SOURCES = ["kernels.cu", "quant.cu", "index_prep.cu", "latent_store.cu", "latent.cu", "latent_api.cu", "api.cu"]
DEPS = SOURCES + ["api_common.h", "kernels.cuh", "latent.cuh", "ptx.cuh", "select.cuh", "wait.cuh"]
HEADER = os.path.join(os.path.dirname(HERE), "include", "fp8idx.h")
# the headers each source includes (its object is rebuilt when one changes)
INCLUDES = {
    "kernels.cu": ["kernels.cuh", "ptx.cuh", "select.cuh", "wait.cuh"],
    "quant.cu": ["ptx.cuh"],
    "index_prep.cu": ["ptx.cuh"],
    "latent_store.cu": ["latent.cuh", "kernels.cuh"],
    "latent.cu": ["latent.cuh", "kernels.cuh", "ptx.cuh", "wait.cuh"],
    "latent_api.cu": ["api_common.h", "kernels.cuh", "latent.cuh"],
    "api.cu": ["api_common.h", "kernels.cuh"],
}


def nvcc_path() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def bind_path() -> str:
    """The compiled Python side of the latent calls.  It holds at::Tensor's layout and this interpreter's
    ABI, so its name carries both: another Python or torch neither loads it nor takes it as built."""
    import torch
    return os.path.join(HERE, f"_bind.{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}.so")


def _newer(target: str, deps) -> bool:
    """Whether `target` is missing or older than one of `deps`."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _bind_stale() -> bool:
    return _newer(bind_path(), [os.path.join(CSRC, "bind.cpp"), HEADER, os.path.abspath(__file__)])


def _stale() -> bool:
    return _newer(LIB, [os.path.join(CSRC, f) for f in DEPS] + [HEADER, os.path.abspath(__file__)]) or _bind_stale()


def build_bind() -> None:
    """Compile csrc/bind.cpp against this interpreter and its torch (host code only)."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    path = bind_path()
    tmp = path + f".tmp{os.getpid()}"
    subprocess.check_call(
        [shutil.which("g++") or "g++", "-std=c++17", "-O2", "-fPIC", "-shared",
         f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
         "-I" + os.path.join(root, "include"), "-I" + os.path.join(cuda, "include"),
         "-I" + sysconfig.get_paths()["include"], "-o", tmp, os.path.join(CSRC, "bind.cpp"),
         "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-ldl"],
        cwd=HERE)
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu (in parallel) into libfp8idx.so (static cudart, no libcuda link)."""
    if not force and not _stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    flags = ["-std=c++17", "-O3", "-lineinfo", "-gencode", "arch=compute_100a,code=sm_100a",
             "-Xcompiler", "-fPIC"]
    if verbose:
        flags.insert(0, "-Xptxas=-v")

    def compile_one(src: str) -> str:
        obj = os.path.join(OBJ, src + ".o")
        deps = [os.path.join(CSRC, f) for f in [src] + INCLUDES[src]] + [HEADER, os.path.abspath(__file__)]
        if force or _newer(obj, deps):
            tmp = obj + f".tmp{os.getpid()}.o"
            subprocess.check_call([nvcc_path(), *flags, "-c", "-o", tmp, os.path.join(CSRC, src)], cwd=HERE)
            os.replace(tmp, obj)
        return obj

    with ThreadPoolExecutor(len(SOURCES) + 1) as pool:
        bind = None
        if force or _bind_stale():
            bind = pool.submit(build_bind)
        objs = list(pool.map(compile_one, SOURCES))
        if bind is not None:
            bind.result()
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-Xcompiler", "-fPIC",
                           "-shared", "-cudart", "static", "-o", tmp, *objs], cwd=HERE)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
