"""Builds libvsa.so (the sm_103a kernels plus the C ABI) in-tree.

Each CUDA translation unit compiles in its own nvcc process (in parallel),
then nvcc links them into ``block_sparse_video_vsa_gb300/_build/libvsa.so``.
Beside them g++ compiles the Python module ``_front`` (csrc/front.cpp) against
the installed PyTorch, under a name with its version; without PyTorch, or where
that fails, the library is built all the same and the cache calls go through
ctypes.  Rebuilds only when a source or header is newer than what was built.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libvsa.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     f"-I{os.path.join(REPO_DIR, 'include')}"]


FRONT_SRC = os.path.join(CSRC, "front.cpp")


def front_path():
    """Where the module for the installed PyTorch and this Python is built; None without PyTorch."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None
    return os.path.join(BUILD_DIR, f"_front-{version}-{sysconfig.get_config_var('SOABI')}.so")


def _front_up_to_date(path) -> bool:
    header = os.path.join(REPO_DIR, "include", "vsa.h")
    return path is None or _newer(path, [FRONT_SRC, header, os.path.abspath(__file__)])


def _try_front(path: str) -> None:
    """_build_front, a failure reported and no module left (an old one may not fit the library)."""
    try:
        _build_front(path)
    except Exception as e:  # whatever it is, the library does not need the module
        if os.path.exists(path):
            os.remove(path)
        sys.stderr.write(f"warning: {os.path.basename(path)} was not built; cache calls go through ctypes "
                         f"(18 to 24 us of the host each, not 2 to 7)\n{e}\n")


def _build_front(path: str) -> None:
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    lib = os.path.join(torch_dir, "lib")
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-I{os.path.join(torch_dir, 'include')}",
           f"-I{sysconfig.get_paths()['include']}", f"-I{os.environ.get('CUDA_HOME', '/usr/local/cuda')}/include",
           f"-I{os.path.join(REPO_DIR, 'include')}", FRONT_SRC, "-o", tmp, f"-L{lib}", f"-Wl,-rpath,{lib}",
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {FRONT_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        [os.path.join(REPO_DIR, "include", "vsa.h"), os.path.abspath(__file__)]


def up_to_date() -> bool:
    """Whether build() would leave everything as it is."""
    return _newer(LIB_PATH, _deps()) and _front_up_to_date(front_path())


def _newer(path, deps) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    front = front_path()
    with ThreadPoolExecutor(max_workers=1) as ex:
        if front is not None and (force or not _front_up_to_date(front)):
            ex.submit(_try_front, front)
        if force or not _newer(LIB_PATH, _deps()):
            _build_library(verbose)
    return LIB_PATH


def _build_library(verbose: bool) -> None:
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(sources())) as ex:
        objs = list(ex.map(compile_one, sources()))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
