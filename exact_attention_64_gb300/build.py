"""Builds libfa2.so (the sm_103a CUDA library behind include/fa2.h) in-tree.

Every CUDA translation unit under csrc/ is compiled by nvcc for sm_103a in
parallel, then linked into exact_attention_64_gb300/libfa2.so. That needs nothing
but CUDA's toolkit. csrc/binding.cpp, the native Python entry points of the
per-token calls, is compiled by g++ beside them and linked against it as
exact_attention_64_gb300/_binding.so, where PyTorch is installed; if that fails the
library is there all the same, a warning says why, and the calls that need the
binding raise. Each is rebuilt only when one of its sources or headers is newer, the
binding also when it was built for another PyTorch or Python.
"""

from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
ROOT = PKG.parent
HEADER = ROOT / "include" / "fa2.h"
BUILD = ROOT / "_build"
LIB = PKG / "libfa2.so"
BINDING = PKG / "_binding.so"
BINDING_FOR = BUILD / "binding_for.txt"  # the PyTorch and Python it was built for
BINDING_ERROR = BUILD / "binding_error.txt"  # why it could not be built

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or "/usr/local/cuda/bin/nvcc"
    return cand if Path(cand).exists() else "nvcc"


def _sources():
    return sorted(CSRC.glob("*.cu"))


def _lib_deps():
    return sorted(CSRC.glob("*.cu")) + sorted(CSRC.glob("*.cuh")) + sorted(CSRC.glob("*.h")) + [HEADER]


def _stale(out: Path, deps) -> bool:
    return not out.exists() or any(p.stat().st_mtime > out.stat().st_mtime for p in deps)


def _torch_tag():
    """What the binding is built for, or None without PyTorch."""
    try:
        import torch
    except ImportError:
        return None
    return f"{torch.__version__} {sys.version}"


def _binding_stale() -> bool:
    tag = _torch_tag()
    if tag is None:
        return False
    return (_stale(BINDING, [CSRC / "binding.cpp", HEADER]) or not BINDING_FOR.exists()
            or BINDING_FOR.read_text() != tag)


def needs_build() -> bool:
    return _stale(LIB, _lib_deps()) or _binding_stale()


def _run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")


def _compile_binding(verbose: bool) -> Path:
    import torch

    inc = Path(torch.__file__).resolve().parent / "include"
    obj = BUILD / "binding.o"
    cuda = Path(_nvcc()).resolve().parent.parent / "include"
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-isystem", str(inc), "-isystem", str(inc / "torch" / "csrc" / "api" / "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", str(cuda),
          "-c", str(CSRC / "binding.cpp"), "-o", str(obj)], "g++ failed on binding.cpp", verbose)
    return obj


def _link_binding(obj: Path, verbose: bool) -> None:
    import torch

    lib = Path(torch.__file__).resolve().parent / "lib"
    tmp = BINDING.with_suffix(".so.tmp")
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", str(tmp), str(obj), f"-L{PKG}", "-lfa2",
          f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
          "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], "link of the binding failed", verbose)
    os.replace(tmp, BINDING)
    BINDING_FOR.write_text(_torch_tag())


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile and link libfa2.so, and the native binding where PyTorch is
    installed; returns the library's path. Raises if the library fails, warns if
    the binding does."""
    lib = force or _stale(LIB, _lib_deps())
    binding = _torch_tag() is not None and (force or _binding_stale())
    if not lib and not binding:
        return LIB
    BUILD.mkdir(exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 1)) as ex:
        binding_obj = ex.submit(_compile_binding, verbose) if binding else None
        if lib:
            _build_lib(ex, verbose)
        if binding:
            BINDING_ERROR.unlink(missing_ok=True)
            try:
                _link_binding(binding_obj.result(), verbose)
            except (RuntimeError, OSError) as e:
                BINDING_ERROR.write_text(str(e))
                warnings.warn(f"the native binding was not built: {e}", RuntimeWarning, stacklevel=2)
    return LIB


def _build_lib(ex, verbose: bool) -> None:
    nvcc = _nvcc()

    def compile_one(src: Path) -> Path:
        obj = BUILD / (src.stem + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", str(src), "-o", str(obj)]
        _run(cmd, f"nvcc failed on {src.name}", verbose)
        return obj

    objs = list(ex.map(compile_one, _sources()))
    tmp = LIB.with_suffix(".so.tmp")
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", str(tmp), *map(str, objs),
           "-Xlinker", "-rpath=/usr/local/cuda/lib64"]
    _run(cmd, "link failed", verbose)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
