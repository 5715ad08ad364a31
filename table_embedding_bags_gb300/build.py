"""In-tree build of libtbe.so for sm_103a (GB300) and of the compiled binding.

Each ``csrc/*.cu`` translation unit is compiled in parallel with nvcc and the
objects are linked into ``table_embedding_bags_gb300/libtbe.so``;
``csrc/marshal.cpp`` becomes ``table_embedding_bags_gb300/_marshal.so``, a
Python module against the installed torch.  Nothing is installed outside the
repository.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libtbe.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.cpp")
MARSHAL = os.path.join(PKG, "_marshal.so")
MARSHAL_STAMP = os.path.join(BUILD, "marshal.stamp")  # what _marshal.so was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libtbe")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "tbe.h")]


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src: str, verbose: bool, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and r.stderr:
        print(r.stderr, file=sys.stderr)
    return obj


def _have_torch() -> bool:
    """Without PyTorch there is nothing to bind to: the library alone is built."""
    try:
        import torch  # noqa: F401
    except ImportError:
        return False
    return True


def _marshal_stamp() -> str:
    import torch

    return f"torch {torch.__version__}, Python {sys.version}, {platform.machine()}"


def _marshal_stale() -> bool:
    """Whether the binding is to be built: from other sources, or against
    another PyTorch or Python, whose C++ interface may not match."""
    if _stale(MARSHAL, [MARSHAL_SRC, os.path.join(INCLUDE, "tbe.h")]) or not os.path.exists(MARSHAL_STAMP):
        return True
    with open(MARSHAL_STAMP) as f:
        return f.read() != _marshal_stamp()


def _compile_marshal(verbose: bool) -> None:
    import torch

    home = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(home, "lib")
    tmp = MARSHAL + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", *[f"-I{d}" for d in include],
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", MARSHAL_SRC, "-o", tmp, f"-L{lib}", "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    os.makedirs(BUILD, exist_ok=True)
    with open(MARSHAL_STAMP, "w") as f:
        f.write(_marshal_stamp())


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if stale) and return the path of libtbe.so."""
    deps = _deps()
    binding = _have_torch() and (force or _marshal_stale())
    if not force and not ptxas_info and not _stale(LIB, deps):
        if binding:
            _compile_marshal(verbose)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        other = ex.submit(_compile_marshal, verbose) if binding else None
        objs = list(ex.map(lambda s: _compile(s, verbose or ptxas_info, extra), srcs))
        if other is not None:
            other.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":  # pragma: no cover
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
