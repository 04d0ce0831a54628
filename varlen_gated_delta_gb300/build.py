"""Build libgdn.so in-tree for sm_103a (GB300).

Every translation unit under csrc/ is compiled by nvcc in parallel with
``-gencode arch=compute_103a,code=sm_103a`` and linked into
``varlen_gated_delta_gb300/libgdn.so`` (static CUDA runtime; the driver API
is reached through the runtime's entry-point query, so no -lcuda).
binding/marshal.cpp, the compiled part of the Python binding, becomes an
extension module beside it that is named for the torch it was built against.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libgdn.so")
MARSHAL_SRC = os.path.join(PKG, "binding", "marshal.cpp")
BUILD_DIR = os.path.join(PKG, "_build")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn.so")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cu", ".cpp")))


def _deps():
    return sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                        if f.endswith((".h", ".cuh"))] + [os.path.join(ROOT, "include", "gdn.h")]


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(d) > t for d in _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [_nvcc(), *ARCH, "-O3", "-std=c++20", "-lineinfo", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd[cmd.index("-c"):cmd.index("-c")] = ["-x", "cu"]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def marshal_path() -> str:
    """The extension module of the running torch and Python."""
    import torch
    tag = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    return os.path.join(PKG, f"_marshal_{sys.implementation.cache_tag}_{tag}.so")


def _build_marshal(force: bool) -> None:
    out = marshal_path()
    deps = [MARSHAL_SRC, os.path.join(ROOT, "include", "gdn.h")]
    if not force and os.path.exists(out) and all(os.path.getmtime(d) <= os.path.getmtime(out) for d in deps):
        return
    if os.path.exists(out):
        os.remove(out)  # (of another source or library: rather none)
    import sysconfig

    import torch
    top = os.path.dirname(torch.__file__)
    lib, inc = os.path.join(top, "lib"), os.path.join(top, "include")
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = out + ".tmp"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *(f"-I{d}" for d in (os.path.join(ROOT, "include"), inc, os.path.join(inc, "torch", "csrc", "api", "include"),
                                sysconfig.get_paths()["include"], os.path.join(cuda, "include"))),
           MARSHAL_SRC, "-o", tmp, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
           "-L", PKG, "-lgdn", f"-Wl,-rpath,{lib}", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MARSHAL_SRC}:\n{r.stderr}")
    os.replace(tmp, out)


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is out of date; returns the library's path.  Where the compiled part of the binding
    cannot be built (it needs g++ and the headers of Python and torch), the library still is: a
    warning tells why, and only the calls that go through that part raise."""
    if force or _stale():
        _build_lib(verbose)
    try:
        _build_marshal(force)
    except (RuntimeError, OSError, ImportError) as e:
        warnings.warn(f"the attention-layer calls have no binding: {e}", RuntimeWarning, stacklevel=2)
    return LIB


def _build_lib(verbose: bool) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-Xlinker", "--no-undefined"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
