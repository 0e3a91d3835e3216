"""Build the sm_100a CUDA library in-tree (nvcc, no JIT cache).

The shared library ``libloza_ssa.so`` is written next to this file so that it
travels with the source tree; it exposes exactly the C ABI of
``include/loza_ssa.h``. Next to it goes ``_paged_binding.so``, the compiled part
of the Python binding (host code against torch's headers, g++).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_PATH = os.path.join(PKG, "libloza_ssa.so")
BINDING_PATH = os.path.join(PKG, "_paged_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "paged_binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libloza_ssa.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [os.path.join(INCLUDE, "loza_ssa.h")])


def up_to_date() -> bool:
    return _newer(LIB_PATH, sources())


def _newer(target: str, inputs) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(s) <= os.path.getmtime(target) for s in inputs)


def _compile(cmd, target: str, verbose: bool):
    """Run a compiler that writes its output file (`{out}` in cmd), and put that in place in one step."""
    tmp = target + f".tmp{os.getpid()}"
    res = subprocess.run([tmp if c == "{out}" else c for c in cmd], capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(os.path.basename(cmd[0]) + " failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stderr)
    os.replace(tmp, target)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/paged_binding.cpp against the installed torch."""
    inputs = [BINDING_SOURCE, os.path.join(INCLUDE, "loza_ssa.h")]
    if not force and _newer(BINDING_PATH, inputs):
        return BINDING_PATH
    import sysconfig
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    system = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
              sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    _compile(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", f"-I{INCLUDE}",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
              f'-DLOZA_TORCH_VERSION="{torch.__version__}"', *[x for d in system for x in ("-isystem", d)],
              "-o", "{out}", BINDING_SOURCE, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
              "-ltorch_python"], BINDING_PATH, verbose)
    return BINDING_PATH


def _build_library(verbose: bool):
    nvcc, units = _nvcc(), sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(os.cpu_count()) as pool:
        objects = [os.path.join(tmp, os.path.basename(u) + ".o") for u in units]
        list(pool.map(lambda u, o: _compile([nvcc, *NVCC_FLAGS, f"-I{INCLUDE}", f"-I{CSRC}", "-c", "-o", "{out}", u],
                                            o, verbose), units, objects))
        _compile([nvcc, *NVCC_FLAGS[:2], "-shared", "-o", "{out}", *objects], LIB_PATH, verbose)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/*.cu into libloza_ssa.so and the binding, each file by a compiler of its own at the same time.

    The library needs nvcc alone. Where the binding cannot be compiled (no g++, Python or torch headers) the entry
    points that do not use it work all the same: a warning says what is missing, and the others raise."""
    with ThreadPoolExecutor(1) as beside:
        binding = beside.submit(build_binding, force, verbose)
        if force or not up_to_date():
            _build_library(verbose)
    try:
        binding.result()
    except (ImportError, OSError, RuntimeError) as e:
        if os.path.exists(BINDING_PATH):  # of another source: its argument structs may not be the library's
            os.remove(BINDING_PATH)
        warnings.warn(f"{os.path.basename(BINDING_PATH)} could not be built, the paged operators are not there: {e}")
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
