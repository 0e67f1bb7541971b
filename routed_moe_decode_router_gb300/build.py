"""Build the CUDA library in-tree: csrc/*.cu -> _build/libmoe_router.so, and
the Python extension that ops.py calls: csrc/ops_binding.cpp -> _build/_moe_ops.so.

nvcc compiles each translation unit for sm_103a in parallel, then links a
shared library against the shared CUDA runtime.  That needs no PyTorch.  g++
compiles the extension against the installed PyTorch and links it to that
library; without PyTorch or Python's headers the library is built alone.
Rebuilds only when a source or header is newer than the results, and the
extension also when it was built for another PyTorch or Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmoe_router.so")
BINDING_SRC = os.path.join(CSRC, "ops_binding.cpp")
BINDING = os.path.join(BUILD, "_moe_ops.so")
BUILT_FOR = BINDING + ".for"     # the PyTorch and Python that the extension was built for
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I", INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return (glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")))


def _newer(result: str, deps) -> bool:
    return os.path.exists(result) and all(os.path.getmtime(d) <= os.path.getmtime(result)
                                          for d in deps)


def target() -> Optional[str]:
    """The PyTorch and Python to build the extension for; None where one of
    them, or Python's headers, is missing."""
    try:
        import torch
    except (ImportError, OSError):
        return None
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return None
    return "PyTorch %s, %s" % (torch.__version__, sysconfig.get_config_var("SOABI"))


def built_for() -> str:
    """What the extension was built for; empty if it never was."""
    try:
        with open(BUILT_FOR) as f:
            return f.read()
    except OSError:
        return ""


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + _headers())


def extension_up_to_date() -> bool:
    return _newer(BINDING, [BINDING_SRC] + _headers()) and built_for() == target()


def _binding_commands():
    """Compile and link commands of the extension, and the file they make."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    obj = os.path.join(BUILD, "ops_binding.o")
    abi = "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi())
    compile_cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", abi,
                   "-I", INCLUDE, "-I", os.path.join(root, "include"),
                   "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                   "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
                   "-c", BINDING_SRC, "-o", obj]
    tmp = BINDING + ".%d.tmp" % os.getpid()
    link_cmd = ["g++", "-shared", "-o", tmp, obj, "-L", BUILD, "-l:libmoe_router.so",
                "-Wl,-rpath,$ORIGIN", "-L", os.path.join(root, "lib"), "-ltorch_python",
                "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10"]
    return compile_cmd, link_cmd, tmp


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, r.stdout, r.stderr))
    return r.stdout + r.stderr


def _build_library(verbose: bool):
    cc = nvcc()
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(src_obj):
        src, obj = src_obj
        log = _run([cc] + NVCC_FLAGS + ["-c", src, "-o", obj], "nvcc on %s" % src)
        if verbose:
            print(log)

    with cf.ThreadPoolExecutor(max_workers=max(1, len(srcs))) as ex:
        list(ex.map(compile_one, zip(srcs, objs)))
    tmp = LIB + ".%d.tmp" % os.getpid()
    _run([cc] + ARCH + ["-shared", "-cudart", "shared", "-Xlinker", "-soname=libmoe_router.so",
                        "-o", tmp] + objs, "link")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date.  Whatever keeps the extension from being
    built, the library is there before this returns or raises."""
    os.makedirs(BUILD, exist_ok=True)
    wanted = target()
    library = force or not library_up_to_date()
    extension = wanted is not None and (force or not extension_up_to_date())
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        if extension:
            compile_cmd, link_cmd, tmp = _binding_commands()
            compiled = ex.submit(_run, compile_cmd, "g++ on %s" % BINDING_SRC)
        if library:
            _build_library(verbose)
        if extension:
            compiled.result()
            _run(link_cmd, "link of the extension")
            os.replace(tmp, BINDING)
            with open(BUILT_FOR, "w") as f:
                f.write(wanted)
    if wanted is None:
        print("built without the extension of ops.py, which needs PyTorch and Python's headers",
              file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
