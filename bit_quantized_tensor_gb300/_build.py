"""Builds libqgemm.so in-tree with nvcc for sm_103a.

Each CUDA translation unit compiles in parallel into ``_build/`` at the
repository root, then nvcc links them into
``bit_quantized_tensor_gb300/libqgemm.so`` with the CUDA runtime linked
statically (the library has no run-time dependency on libcudart or
libcuda; the driver's tensor-map encoder is fetched through the runtime's
entry-point query).  Beside it g++ builds ``_qg_host.so``, the torch-facing
host side of the small calls, where a torch with CUDA is installed; the library
needs neither.  Each of the two is built only when it is older than its sources
and headers, and the second also when torch or Python has changed.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqgemm.so")
HOST_SRC = os.path.join(CSRC, "qg_host.cpp")
HOST = os.path.join(PKG, "_qg_host.so")
HOST_FOR = os.path.join(BUILD_DIR, "_qg_host.for")  # what HOST was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-O2", "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libqgemm.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(out: str, deps: list[str]) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps)


def _headers() -> list[str]:
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + _headers())


def _installed() -> str:
    """The torch and Python that the extension is built against; empty without torch."""
    if importlib.util.find_spec("torch") is None:
        return ""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "unknown"
    return f"torch {torch}, Python {sys.version_info.major}.{sys.version_info.minor}"


def host_up_to_date() -> bool:
    """True also where there is nothing to build it against."""
    now = _installed()
    if not now:
        return True
    try:
        with open(HOST_FOR) as f:
            built = f.read()
    except OSError:
        built = ""
    return built in (now, now + NO_CUDA) and (built != now or _newer(HOST, [HOST_SRC] + _headers()))


def up_to_date() -> bool:
    return library_up_to_date() and host_up_to_date()


NO_CUDA = ", without CUDA"


def build_host() -> None:
    """The Python extension of csrc/qg_host.cpp, against the torch that is installed."""
    import sysconfig

    import torch
    os.makedirs(BUILD_DIR, exist_ok=True)
    if torch.version.cuda is None:
        with open(HOST_FOR, "w") as f:
            f.write(_installed() + NO_CUDA)
        return
    tdir = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = HOST + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-o", tmp, HOST_SRC, "-I", INCLUDE,
           "-I", os.path.join(tdir, "include"), "-I", os.path.join(tdir, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-L", os.path.join(tdir, "lib"), "-lc10", "-ltorch_cpu", "-lc10_cuda", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {HOST_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, HOST)
    with open(HOST_FOR, "w") as f:
        f.write(_installed())


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is out of date; a failure of the extension is raised once the library is there."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        host = None
        if _installed() and (force or not host_up_to_date()):
            host = ex.submit(build_host)
        if force or not library_up_to_date():
            build_library(verbose)
        if host is not None:
            host.result()
    return LIB


def build_library(verbose: bool = False) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + NVCC_FLAGS + ["-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
