"""Build libvgqa.so (the C ABI in include/varlen_gqa.h) for sm_100a with nvcc.

    python -m varlen_gqa_split_b200.build [--force]

Compiles each source to an object in parallel, then links one shared library
into varlen_gqa_split_b200/_lib/ (in-tree).  Only the attn_* symbols are
exported (-fvisibility=hidden).  cudart is linked statically so the library
does not depend on the runtime version another component of the process
loaded.  Rebuilds only when a source or header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(HERE, "_build")
LIBDIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIBDIR, "libvgqa.so")
# the binding's native marshalling (a Python extension module; needs torch's
# headers, calls the library through its C ABI)
MARSHAL_SRC = os.path.join(CSRC, "python", "marshal.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-I", INCLUDE,
                     "-Xcompiler", "-fPIC,-fvisibility=hidden", "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _deps())


def marshal_path() -> str:
    """The module for the torch and the interpreter that run: another torch
    gets another one."""
    from ._binding import MARSHAL_PATH
    return MARSHAL_PATH


def marshal_up_to_date() -> bool:
    path = marshal_path()
    deps = [MARSHAL_SRC, os.path.join(INCLUDE, "varlen_gqa.h"), os.path.abspath(__file__)]
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in deps)


def build_marshal() -> str:
    import sysconfig

    import torch
    base = os.path.join(os.path.dirname(torch.__file__))
    inc = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include")]
    path = marshal_path()
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"] + [f"-I{d}" for d in inc] + \
        [MARSHAL_SRC, "-o", tmp, "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def _compile(src: str, verbose: bool) -> tuple[str, str]:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [nvcc()] + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr if verbose else ""


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libvgqa.so and the binding's marshalling module;
    returns the library's path."""
    os.makedirs(LIBDIR, exist_ok=True)
    if not force and up_to_date():
        if not marshal_up_to_date():
            build_marshal()
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        module = ex.submit(build_marshal) if force or not marshal_up_to_date() else None
        results = list(ex.map(lambda s: _compile(s, verbose), sources()))
        if module:
            module.result()
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in results] + ["-lcuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        # libcuda is only needed for symbol resolution of the driver entry
        # point typedefs; link without it if the stub is not on the path
        cmd = cmd[:-1]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
