"""Build the CUDA library ``_lib/libpkv.so`` in-tree for sm_103a.

Each ``csrc/*.cu`` file is compiled by nvcc in parallel, then linked into one
shared library with the CUDA runtime linked statically; beside them the host
compiler builds ``_lib/_calls.<interpreter>-torch<version>.so``
(``csrc/calls.cpp``), the Python binding's argument checks for the E2M1 calls,
against this interpreter and its torch.  Rebuilds the one or the other only when it
is missing or a source or header of it is newer.  The library needs nvcc alone:
without torch, its headers or Python's the checks are left out (with a warning where
there is a torch to bind), and the E2M1 calls from Python raise.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libpkv.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def calls_path() -> str:
    """The compiled argument checks for this interpreter and this torch (their ABI
    is in the name: another one's are never loaded)."""
    import torch
    tag = f"{sysconfig.get_config_var('SOABI')}-torch{torch.__version__}"
    return os.path.join(OUT_DIR, f"_calls.{tag}.so")


def _older(built: str, deps) -> bool:
    return not os.path.exists(built) or any(os.path.getmtime(p) > os.path.getmtime(built)
                                            for p in deps)


def _stale() -> bool:
    return _older(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _calls_stale(force: bool) -> bool:
    try:
        return _older(calls_path(), [os.path.join(CSRC, "calls.cpp")]) or force
    except ImportError:                                  # no torch: nothing to bind
        return False


def _build_calls() -> None:
    """Compile the argument checks of the E2M1 calls against torch's headers."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    calls = calls_path()
    tmp = calls + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "calls.cpp"),
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, calls)


def _try_build_calls() -> None:
    try:
        _build_calls()
    except (RuntimeError, OSError) as e:
        warnings.warn(f"the E2M1 calls are not available from Python: {e}", RuntimeWarning)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library, and the binding's argument checks, if needed;
    return the library's path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    calls_stale = _calls_stale(force)
    if not force and not _stale():
        if calls_stale:
            _try_build_calls()
        return LIB
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        calls = ex.submit(_try_build_calls) if calls_stale else None
        objs = list(ex.map(compile_one, _sources()))
        if calls is not None:
            calls.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
