"""Builds libattn_gb300.so from csrc/ with nvcc for sm_103a (in-tree, no setuptools), and beside it the compiled part of
the Python binding (csrc/calls.cpp, against torch's headers). The library needs neither torch nor that part: without torch it
is built alone, and it is linked before a failing compilation of calls.cpp is reported.

Each .cu file compiles in its own nvcc process (in parallel); the objects are linked into one
shared library next to this file. The CUDA runtime is linked statically and the driver's
tensor-map encoder is looked up at run time, so the library loads on machines without a GPU
driver (the ABI tests check its exports there).
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_NAME = "libattn_gb300.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
EXT_SUFFIX = sysconfig.get_config_var("EXT_SUFFIX")
CALLS_PATH = os.path.join(PKG_DIR, "_calls" + EXT_SUFFIX)
CALLS_STAMP = os.path.join(BUILD_DIR, "calls.txt")   # the environment that CALLS_PATH was built for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch_dir() -> Optional[str]:
    """Where torch is installed; None without torch."""
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec else None


def has_torch() -> bool:
    return _torch_dir() is not None


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + _headers()


def _newer(path: str, deps) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in deps)


def _library_up_to_date() -> bool:
    return _newer(LIB_PATH, _deps())


def _calls_up_to_date() -> bool:
    return _newer(CALLS_PATH, [os.path.join(CSRC, "calls.cpp")] + _headers()) and calls_fit()


def up_to_date() -> bool:
    return _library_up_to_date() and (not has_torch() or _calls_up_to_date())


def _environment() -> str:
    """What the compiled calls are bound to: the interpreter's ABI, and one torch by its place and version."""
    torch_dir = _torch_dir()
    with open(os.path.join(torch_dir, "version.py")) as f:
        return "\n".join([EXT_SUFFIX, torch_dir, f.read()])


def calls_fit() -> bool:
    """Whether the compiled calls were built for the interpreter and torch that run now."""
    if not os.path.exists(CALLS_STAMP):
        return False
    with open(CALLS_STAMP) as f:
        return f.read() == _environment()


def _compile(nvcc: str, src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_calls(nvcc: str) -> str:
    obj = os.path.join(BUILD_DIR, "calls.o")
    includes = [os.path.join(_torch_dir(), "include"), sysconfig.get_paths()["include"],
                os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include"), INCLUDE]
    _run(["g++", "-O2", "-std=c++17", "-fPIC"] + ["-I" + p for p in includes] +
         ["-c", os.path.join(CSRC, "calls.cpp"), "-o", obj], "g++ for calls.cpp")
    return obj


def _link_library(nvcc: str, objs) -> None:
    tmp = LIB_PATH + ".tmp"
    _run([nvcc] + ARCH + ["-shared", "-Xlinker", "-soname=" + LIB_NAME, "-o", tmp] + objs, "link")
    os.replace(tmp, LIB_PATH)


def _link_calls(obj: str) -> None:
    # finds the library beside itself, and torch's where they were when it was built
    torch_lib, tmp, stamp = os.path.join(_torch_dir(), "lib"), CALLS_PATH + ".tmp", CALLS_STAMP + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG_DIR, "-l:" + LIB_NAME, "-L" + torch_lib, "-ltorch_python",
          "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib],
         "link of the compiled calls")
    with open(stamp, "w") as f:
        f.write(_environment())
    os.replace(tmp, CALLS_PATH)
    os.replace(stamp, CALLS_STAMP)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles (what is not up to date) and returns the path of the shared library."""
    library = force or not _library_up_to_date()
    calls = has_torch() and (force or not _calls_up_to_date())
    if not library and not calls:
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources() if library else []
    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        calls_obj = ex.submit(_compile_calls, nvcc) if calls else None
        objs = list(ex.map(lambda s: _compile(nvcc, s, verbose), srcs))
    if library:
        _link_library(nvcc, objs)
    if calls:
        _link_calls(calls_obj.result())
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
