"""Builds libmedusa_gb300.so in-tree for sm_103a (nvcc, one -gencode).

Each translation unit is compiled in parallel to an object file, then linked
into one shared library with the CUDA runtime linked statically, so the library
loads on a machine without a GPU (entry points then return MEDUSA_ERR_CUDA).

Where torch is installed, the compiled bindings of the calls that are made once per
layer (csrc/python) are built beside it, against that torch's headers.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.machinery
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmedusa_gb300.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmedusa_gb300")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps() -> list:
    return sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _newer(target: str, deps: list) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


BINDINGS = ("paged_binding", "verify_binding")


def binding_path(name: str = BINDINGS[0]) -> str:
    """The compiled binding for this Python (version, platform) and the installed
    torch (version, C++ ABI)."""
    import torch
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(BUILD, f"{name}-{torch.__version__}-abi{abi}{sysconfig.get_config_var('EXT_SUFFIX')}")


def load_binding(name: str):
    """The compiled binding as a module (raises if it has not been built)."""
    path = binding_path(name)
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} does not exist: run medusa_head_speculative_heads_gb300.build.build() first")
    spec = importlib.util.spec_from_loader(name, importlib.machinery.ExtensionFileLoader(name, path))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def build_binding(force: bool = False) -> None:
    """Compiles csrc/python against the installed torch (nothing without one) and
    links it to the library, which lies beside it."""
    try:
        import torch
    except ImportError:
        return
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    deps = glob.glob(os.path.join(CSRC, "python", "*.h")) + [os.path.join(INCLUDE, "medusa.h")]

    def compile_one(name):
        src, out = os.path.join(CSRC, "python", f"{name}.cpp"), binding_path(name)
        if not force and _newer(out, [src] + deps):
            return
        tmp = out + f".{os.getpid()}.tmp"
        cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", src, "-o", tmp]
        for d in (INCLUDE, f"{t}/include", f"{t}/include/torch/csrc/api/include", f"{cuda}/include", sysconfig.get_paths()["include"]):
            cmd += ["-I", d]
        cmd += [f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-L{t}/lib", "-ltorch_python", "-ltorch_cpu",
                "-lc10_cuda", "-lc10", f"-L{BUILD}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{name} does not build:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, out)

    with cf.ThreadPoolExecutor(len(BINDINGS)) as ex:
        list(ex.map(compile_one, BINDINGS))


def build(force: bool = False, verbose: bool = False, extra_flags: list | None = None) -> str:
    if not force and up_to_date():
        build_binding()
        return LIB
    os.makedirs(os.path.join(BUILD, "obj"), exist_ok=True)
    cc = nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
                     "--expt-relaxed-constexpr"] + list(extra_flags or [])

    def compile_one(src):
        obj = os.path.join(BUILD, "obj", os.path.basename(src) + ".o")
        cmd = [cc, "-c", src, "-o", obj] + common
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with cf.ThreadPoolExecutor(max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
