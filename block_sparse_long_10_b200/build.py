"""Build libqsa.so in-tree with nvcc for sm_100a (B200).

Each ``csrc/*.cu`` file is compiled to an object under ``_build/`` (in
parallel, skipped when up to date) and linked, with the CUDA runtime linked
statically, into ``block_sparse_long_10_b200/libqsa.so``.  ``csrc/bind.cpp``, the
native part of the Python binding, becomes ``_bind.so`` beside it (g++, against
torch's headers; left out where there is no torch with CUDA).
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqsa.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(PKG, "_bind.so")
BIND_STAMP = os.path.join(BUILD, "bind.stamp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", os.path.join(ROOT, "include"),
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps_mtime() -> float:
    files = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    files.append(os.path.join(ROOT, "include", "qsa.h"))
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, extra: list[str], verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    if (os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
            and os.path.getmtime(obj) >= _deps_mtime()):
        return obj
    cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr.strip():
        print(r.stderr, file=sys.stderr)
    return obj


def build(verbose: bool = False, extra: list[str] | None = None, force: bool = False) -> str:
    """Compile every CUDA source and link libqsa.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    extra = list(extra or [])
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra, verbose), srcs))
    if not (os.path.exists(LIB)
            and os.path.getmtime(LIB) >= max(os.path.getmtime(o) for o in objs)):
        _link([_nvcc(), *ARCH, "-shared", "-cudart", "static", *objs], LIB, verbose)
    _build_bind(verbose)
    return LIB


def _build_bind(verbose: bool) -> None:
    """The Python binding's native part, where there is a CUDA build of torch to make it
    against (the C library does not need one); made again when that torch, or the Python,
    is another one."""
    made_for = _bind_made_for()
    newest = max(os.path.getmtime(f) for f in (BIND_SRC, os.path.join(ROOT, "include", "qsa.h")))
    if os.path.exists(BIND) and os.path.getmtime(BIND) >= newest and made_for is not None:
        with contextlib.suppress(FileNotFoundError), open(BIND_STAMP) as f:
            if f.read() == made_for:
                return
    if made_for is None:
        print(f"{BIND} is not built: no torch with CUDA", file=sys.stderr)
        with contextlib.suppress(FileNotFoundError):
            os.remove(BIND)  # one for another torch does not load, or worse
        return
    _link(_bind_cmd(), BIND, verbose)
    with open(BIND_STAMP, "w") as f:
        f.write(made_for)


def _bind_made_for() -> str | None:
    """The torch and Python that a binding built now is for; None without a usable torch."""
    try:
        import torch
    except ImportError:
        return None
    home = os.path.dirname(torch.__file__)
    for f in ("include/c10/cuda/CUDAStream.h", "lib/libc10_cuda.so", "lib/libtorch_python.so"):
        if not os.path.exists(os.path.join(home, f)):
            return None
    return (f"{torch.__version__} cxx11abi={int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"{sysconfig.get_config_var('SOABI')}")


def _link(cmd: list[str], out: str, verbose: bool) -> None:
    tmp = out + f".tmp{os.getpid()}"
    cmd = [*cmd, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {out} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _bind_cmd() -> list[str]:
    import torch

    home = os.path.dirname(torch.__file__)
    inc = [os.path.join(home, "include"), os.path.join(home, "include/torch/csrc/api/include"),
           os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),
           sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-I{i}" for i in inc), BIND_SRC, f"-L{PKG}", "-l:libqsa.so", "-Wl,-rpath,$ORIGIN",
            f"-L{os.path.join(home, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
            "-lc10"]


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(verbose=v, extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else None,
                force="--force" in sys.argv))
