"""Build libq8.so (the CUDA library behind include/q8.h) in place, for sm_103a only.

Each .cu file under csrc/ is compiled in parallel with nvcc
(``-gencode arch=compute_103a,code=sm_103a``, no fast-math, IEEE division and
square root) and linked into ``q8_quantized_matmul_gb300/libq8.so`` with the
CUDA runtime linked statically, so loading the library needs no GPU.
``csrc/q8_torch.cpp`` becomes ``_q8torch.so`` beside it (g++, torch's headers) where torch is installed: the C
library needs nvcc alone.

    python -m q8_quantized_matmul_gb300.build
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libq8.so")
HEADER = os.path.join(ROOT, "include", "q8.h")
TORCH_EXT = os.path.join(PKG, "_q8torch.so")   # csrc/q8_torch.cpp: the tensor helpers' marshalling

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
# No fast-math: '/' must be the IEEE division and subnormals must be kept
# (the quantiser is bit-exact to the CPU definition).
NVFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-prec-div=true", "-prec-sqrt=true",
           "-fmad=true", "-ftz=false"]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libq8.so")
    return exe


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _newer(out: str, files: list[str]) -> bool:
    """Whether one of the files is newer than `out`, or there is no such file."""
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(f) > t for f in files)


def torch_version() -> str | None:
    """The installed torch's version (not imported for it), or None."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:   # a source tree on the path has no metadata
        return "of a source tree" if importlib.util.find_spec("torch") else None


def lib_stale() -> bool:
    return _newer(LIB, [HEADER] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != "q8_torch.cpp"])


def ext_stale() -> bool:
    """Whether the tensor helpers' module is to be built: never without torch, again for another one."""
    version = torch_version()
    if version is None:
        return False
    if _newer(TORCH_EXT, [HEADER, os.path.join(CSRC, "q8_torch.cpp")]):
        return True
    try:
        with open(os.path.join(OBJ, "torch_version")) as f:
            return f.read() != f"{version} python {sys.version}"
    except OSError:
        return True


def stale() -> bool:
    return lib_stale() or ext_stale()


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVFLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_torch() -> None:
    """The CPython module of the tensor helpers, against the installed torch's headers and libraries."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    tmp = TORCH_EXT + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O1", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", sysconfig.get_paths()["include"],
           "-isystem", cuda, os.path.join(CSRC, "q8_torch.cpp"), "-o", tmp, f"-L{lib}", "-lc10", "-ltorch_cpu",
           "-lc10_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for q8_torch.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_EXT)


def _link(objs: list[str]) -> None:
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _build_ext() -> None:
    _compile_torch()
    with open(os.path.join(OBJ, "torch_version"), "w") as f:
        f.write(f"{torch_version()} python {sys.version}")


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    """Compile what is older than its sources (or all, with force): libq8.so, and with torch installed _q8torch.so.
    An error of the latter is raised once libq8.so is in place."""
    lib, ext = force or lib_stale(), torch_version() is not None and (force or ext_stale())
    if not (lib or ext):
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        helpers = ex.submit(_build_ext) if ext else None
        if lib:
            _link(list(ex.map(lambda s: _compile(s, extra), srcs)))
        if helpers:
            helpers.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
