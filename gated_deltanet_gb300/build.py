"""Build the sm_103a shared library ``libgdn.so`` in-tree with nvcc.

Each ``csrc/*.cu`` file is compiled to an object in parallel (one -gencode,
sm_103a only) and linked into ``gated_deltanet_gb300/_lib/libgdn.so``.
Beside it, ``csrc/layer_binding.cpp`` (the compiled part of the Python binding) becomes ``_lib/_layer.so``
with the host compiler, against the installed PyTorch's headers; without PyTorch the library alone is built.  A rebuild
happens only when a source or header is newer than what was built, and for the binding when PyTorch or Python is
another than it was built for.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libgdn.so")
BINDING_SRC = os.path.join(CSRC, "layer_binding.cpp")
BINDING = os.path.join(LIBDIR, "_layer.so")
BUILT_FOR = os.path.join(LIBDIR, "_layer.built_for")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "gdn.h"), os.path.abspath(__file__)]


def lib_path() -> str:
    return LIB


def binding_path() -> str:
    return BINDING


def running() -> str | None:
    """What the binding has to be built for: this PyTorch and this Python; None without PyTorch."""
    try:
        import torch
    except ImportError:
        return None
    return f"torch {torch.__version__}, python {sys.version_info[0]}.{sys.version_info[1]}"


def built_for() -> str | None:
    """What the binding was built for; None where none was."""
    try:
        with open(BUILT_FOR) as f:
            return f.read()
    except FileNotFoundError:
        return None


def _stale(built: str, deps) -> bool:
    return not os.path.exists(built) or any(os.path.getmtime(p) > os.path.getmtime(built) for p in deps)


def _binding_stale() -> bool:
    now = running()
    return now is not None and (built_for() != now or _stale(BINDING, _deps() + [BINDING_SRC]))


def needs_build() -> bool:
    return _stale(LIB, _deps()) or _binding_stale()


def _compile_binding() -> str:
    """The binding's object file (its library is linked once ``libgdn.so`` exists)."""
    import sysconfig

    import torch

    t = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(OBJ, "layer_binding.o")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", t, "-isystem", os.path.join(t, "torch", "csrc", "api", "include"), "-isystem", cuda,
           "-isystem", sysconfig.get_paths()["include"], "-I", os.path.join(ROOT, "include"), "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch

    t = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, LIB, "-Wl,-rpath,$ORIGIN", "-L" + t, "-ltorch_python", "-ltorch_cpu",
           "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {BINDING} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BUILT_FOR + f".tmp{os.getpid()}", "w") as f:
        f.write(running())
    os.replace(f.name, BUILT_FOR)


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    library, binding = force or _stale(LIB, _deps()), running() is not None and (force or _binding_stale())
    if not library and not binding:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                    "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc()] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    srcs = _sources() if library else []
    with ThreadPoolExecutor(max_workers=jobs or min(12, len(srcs) + 1)) as ex:
        obj = ex.submit(_compile_binding) if binding else None
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for _, err in results:
            if err:
                print(err)
    if library:
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc()] + ARCH + ["-shared", "-Xlinker", "-soname=libgdn.so", "-o", tmp] + [o for o, _ in results] + ["-lcudart_static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if binding:  # (last: what fails here does not cost the library)
        _link_binding(obj.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
