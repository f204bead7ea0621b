"""In-tree build of libnvfp4moe.so for sm_103a with nvcc (no cmake).

Each .cu file under csrc/ is compiled in parallel to an object with
``-gencode arch=compute_103a,code=sm_103a``, then linked into one shared
library (static CUDA runtime) next to this file.  csrc/torch_calls.cpp, the
host side of the short operators on torch's tensors, becomes an extension
module linked to that library; where torch or its headers are missing, the
library is built alone.  Each is rebuilt when a source or header of its own is
newer than it, the extension also when torch or Python is another one.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnvfp4moe.so")
EXT_SRC = os.path.join(CSRC, "torch_calls.cpp")
EXT = os.path.join(PKG, "_torch_calls.so")
EXT_FOR = os.path.join(BUILD, "torch_calls.for")  # the torch and Python that EXT was built for
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libnvfp4moe")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def lib_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  _headers())


def torch_dir():
    """Where torch lies, None without torch or its headers (found without importing it)."""
    spec = importlib.util.find_spec("torch")
    where = os.path.dirname(spec.origin) if spec and spec.origin else None
    return where if where and os.path.exists(os.path.join(where, "include", "ATen", "ATen.h")) else None


def _ext_for(where) -> str:
    with open(os.path.join(where, "version.py")) as f:
        return f"{where}\n{sys.version}\n{f.read()}"


def ext_up_to_date(where) -> bool:
    if not _newer(EXT, [EXT_SRC] + _headers()) or not os.path.exists(EXT_FOR):
        return False
    with open(EXT_FOR) as f:
        return f.read() == _ext_for(where)


def up_to_date() -> bool:
    where = torch_dir()
    return lib_up_to_date() and (where is None or ext_up_to_date(where))


def _compile(src, extra):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", obj] + extra
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_ext():
    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(BUILD, "torch_calls.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = [f"-I{d}" for d in cpp_extension.include_paths() + [cuda, sysconfig.get_paths()["include"]]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", EXT_SRC, "-o", obj,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + inc
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on torch_calls.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_ext(obj):
    from torch.utils import cpp_extension
    tmp = EXT + ".tmp"
    cmd = ["g++", "-shared", obj, "-o", tmp] + [f"-L{d}" for d in cpp_extension.library_paths() + [PKG]] + [
        "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-ltorch_python", "-l:libnvfp4moe.so",
        "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)


def _link_lib(objs):
    tmp = LIB + ".tmp"
    cmd = [nvcc(), ARCH, "-shared", "-Xlinker", "-soname=libnvfp4moe.so", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libnvfp4moe.so, and torch's extension where there is torch; returns the library's path."""
    where = torch_dir()
    lib = force or not lib_up_to_date()
    ext = where is not None and (force or not ext_up_to_date(where))
    if not lib and not ext:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        ext_obj = ex.submit(_compile_ext) if ext else None
        if lib:
            results = list(ex.map(lambda s: _compile(s, list(extra_flags)), sources()))
            if verbose:
                for _, log in results:
                    if log.strip():
                        print(log, file=sys.stderr)
            _link_lib([o for o, _ in results])
        if ext:
            _link_ext(ext_obj.result())
            with open(EXT_FOR, "w") as f:
                f.write(_ext_for(where))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
