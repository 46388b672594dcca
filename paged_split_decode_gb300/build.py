"""Build libpdecode.so in-tree with nvcc for sm_103a.

Each translation unit under csrc/ is compiled in parallel to an object file
under _build/, then linked into paged_split_decode_gb300/libpdecode.so (the
CUDA runtime is linked statically; the driver's tensor-map encoder is reached
through the runtime's entry-point query, so no -lcuda is needed). csrc/bind.cpp
becomes _bind.so beside it, the compiled part of the Python binding, against
the headers of the installed PyTorch. The library does not depend on it: where
those headers are missing the library is built all the same, with a warning, and
the calls that go through the compiled binding raise. Each of the two is built
when it is older than a source or header of its own, _bind.so also when PyTorch
is not the one it was built for.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libpdecode.so")
BIND = os.path.join(PKG, "_bind.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND_FOR = os.path.join(BUILD, "bind.for")  # the PyTorch and Python that _bind.so was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpdecode")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _bind_for() -> str:
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "missing"
    return f"torch {version} python {sys.version.split()[0]}"


def _bind_command(out: str):
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    lib = os.path.join(torch_dir, "lib")
    return [nvcc(), "-O2", "-std=c++17", "-shared", "-Xcompiler", "-fPIC,-fvisibility=hidden,-w",
            "-I", os.path.join(ROOT, "include"), "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(torch_dir, "include"), BIND_SRC, "-o", out, "-L", lib, "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_python", "-Xlinker", f"-rpath={lib}"]


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in [*deps, *glob.glob(os.path.join(ROOT, "include", "*.h")), __file__])


def _stale() -> bool:
    headers = glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
    return _older(LIB, sources() + headers)


def _bind_stale() -> bool:
    if not os.path.exists(BIND_FOR) or open(BIND_FOR).read() != _bind_for():
        return True
    return _older(BIND, [BIND_SRC])


def _build_bind() -> str:
    """Build _bind.so; returns "" or what failed."""
    tmp = BIND + f".tmp{os.getpid()}"
    try:
        r = subprocess.run(_bind_command(tmp), capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(tmp, BIND)
            with open(BIND_FOR, "w") as f:
                f.write(_bind_for())
            return ""
        why = f"{r.stdout}\n{r.stderr}"
    except (OSError, AttributeError) as e:  # no compiler, no PyTorch
        why = repr(e)
    if os.path.exists(BIND):
        os.remove(BIND)  # one of other sources or another PyTorch
    return why


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    lib, bind = force or _stale(), force or _bind_stale()
    if not lib and not bind:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 1)) as ex:
        bind_done = ex.submit(_build_bind) if bind else None
        if lib:
            objs = list(ex.map(compile_one, sources()))
            tmp = LIB + f".tmp{os.getpid()}"
            r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, LIB)
        why = bind_done.result() if bind_done else ""
    if why:
        warnings.warn(f"build of {BIND_SRC} failed; the calls of the compiled binding will raise:\n{why}",
                      RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
