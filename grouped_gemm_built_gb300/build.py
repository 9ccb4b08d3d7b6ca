"""Build the sm_103a shared library libmok.so in-tree (grouped_gemm_built_gb300/_lib/).

Every CUDA translation unit under csrc/ is compiled in parallel with nvcc for
``-gencode arch=compute_103a,code=sm_103a`` and linked into one shared library with a
C ABI (include/mok.h, mok_ops.h). csrc/torch_calls.cpp becomes the Python module mok_torch
beside it (g++ against the installed torch's headers). No CMake; the whole build takes well
under a minute.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB_NAME = "libmok.so"
TORCH_NAME = "mok_torch.so"

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    p = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(p):
        return p
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def lib_path() -> str:
    return os.path.join(OUT_DIR, LIB_NAME)


def torch_lib_path() -> str:
    return os.path.join(OUT_DIR, TORCH_NAME)


def torch_tag() -> str:
    """What mok_torch is compiled against: the installed torch, its C++ ABI and this Python's."""
    import torch

    return (f"{torch.__version__} abi{int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"{sysconfig.get_config_var('SOABI')} {os.path.dirname(torch.__file__)}")


def torch_calls_tag() -> str:
    """The tag that the mok_torch in the tree was built with ("" without one)."""
    try:
        with open(torch_lib_path() + ".tag") as f:
            return f.read()
    except OSError:
        return ""


def _build_torch_calls(target: str) -> None:
    """csrc/torch_calls.cpp -> the extension module mok_torch, for the installed torch."""
    import torch

    root = os.path.dirname(torch.__file__)
    inc = [os.path.join(root, "include"), os.path.join(root, "include/torch/csrc/api/include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"),
           sysconfig.get_paths()["include"], os.path.join(ROOT, "include")]
    libs = os.path.join(root, "lib")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in inc), os.path.join(CSRC, "torch_calls.cpp"), "-o", target + ".tmp",
           f"-L{libs}", f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
           "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for torch_calls.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(target + ".tmp", target)
    with open(target + ".tag", "w") as f:
        f.write(torch_tag())


def _needs_build(objs_src, target):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    inc = os.path.join(ROOT, "include")
    deps = list(objs_src) + [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps += [os.path.join(inc, f) for f in os.listdir(inc) if f.endswith(".h")]
    deps.append(os.path.abspath(__file__))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    srcs = sources()
    target = lib_path()
    if not force and not _needs_build(srcs, target) and not _needs_build(srcs, torch_lib_path()):
        if torch_calls_tag() != torch_tag():      # another torch than it was built for
            _build_torch_calls(torch_lib_path())
        return target
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        calls = ex.submit(_build_torch_calls, torch_lib_path())
        objs = list(ex.map(compile_one, srcs))
    tmp = target + ".tmp"
    # No -lcuda: the tensor-map encoder is fetched through the runtime's driver entry
    # points, so the library loads on machines without a driver too.
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, target)
    calls.result()      # last: the C library does not depend on torch or its headers
    return target


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
