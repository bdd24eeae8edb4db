"""Build ``libfm.so`` in-tree with nvcc for sm_103a, and ``_fmcache.so``, the
Python module of the paged cache's calls.

Each ``csrc/*.cu`` compiles to ``_build/<name>.o`` in parallel, then one
nvcc link makes the shared library next to this file.  ``csrc/fm_binding.cpp``
compiles with the host compiler against torch's headers and links to the
library.  Rebuilds only when a source or header is newer than its result, and the
module also when it was built against another torch.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libfm.so")
BINDING = os.path.join(CSRC, "fm_binding.cpp")
MODULE = os.path.join(PKG, "_fmcache.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.isabs(c) and os.path.exists(c) or not os.path.isabs(c)):
            return c
    return "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) \
        + glob.glob(os.path.join(INCLUDE, "*.h"))


def _newer(result, deps) -> bool:
    if not os.path.exists(result):
        return False
    t = os.path.getmtime(result)
    return all(os.path.getmtime(f) <= t for f in deps)


def _binding_deps():
    return [BINDING, os.path.join(INCLUDE, "fm.h")]


def _torch_version():
    try:
        import torch
    except ImportError:
        return None
    return torch.__version__


def _binding_stamp():
    """The file that holds the torch version that the module was built against."""
    return os.path.join(BUILD, "fm_binding.torch")


def _lib_up_to_date() -> bool:
    return _newer(LIB, _deps())


def _binding_up_to_date() -> bool:
    if not _newer(MODULE, _binding_deps()) or not os.path.exists(_binding_stamp()):
        return False
    with open(_binding_stamp()) as f:
        return f.read() == _torch_version()


def up_to_date() -> bool:
    return _lib_up_to_date() and _binding_up_to_date()


def _compile_binding(obj):
    import sysconfig

    import torch
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    inc = [base, os.path.join(base, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
           cuda, INCLUDE]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          *(a for i in inc for a in ("-isystem", i)), "-c", BINDING, "-o", obj], "the binding")


def _link_binding(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MODULE + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libfm.so", "-L" + libs, "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "linking the binding")
    os.replace(tmp, MODULE)
    with open(_binding_stamp(), "w") as f:
        f.write(torch.__version__)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _build_lib(ex, verbose):
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + ".tmp"
    # no -lcuda: the TMA encoder is fetched through the runtime's driver
    # entry-point query, so the library loads on machines without a driver
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], "linking the library")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link what is not up to date; returns the path of the shared library.

    The library comes first and needs nvcc only.  Where the Python module cannot be
    built (no g++, Python.h or torch headers), the call raises after the library is in
    place."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    binding = os.path.join(BUILD, "fm_binding.o")
    with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        made = ex.submit(_compile_binding, binding) if force or not _binding_up_to_date() else None
        if force or not _lib_up_to_date():
            _build_lib(ex, verbose)
        if made:
            made.result()
            _link_binding(binding)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
