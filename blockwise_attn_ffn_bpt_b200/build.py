"""Build the CUDA library libbpt.so in-tree for sm_100a, and the part of the
Python binding that is C++ (csrc/binding.cpp, linked with it).

    python -m blockwise_attn_ffn_bpt_b200.build [--force] [--verbose]

Without torch the library alone is built (python blockwise_attn_ffn_bpt_b200/build.py:
the package itself imports torch).

nvcc cross-compiles without a GPU. The library links the CUDA runtime
statically and reaches the driver's tensor-map encoder through the runtime's
driver entry-point query, so it needs no libcuda at link time.
"""

from __future__ import annotations

import argparse
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libbpt.so")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BUILT_FOR = os.path.join(PKG, "_binding.torch")  # the torch that BINDING was built against

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-Xptxas", "-v",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "bpt.h")])


def up_to_date() -> bool:
    return _newer(LIB, sources()) and (installed_torch() is None or binding_up_to_date())


def installed_torch():
    """The installed torch, as a text that another one has not; None where there is none."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "?"
    return f"{version} {spec.origin}"


def binding_up_to_date() -> bool:
    if not _newer(BINDING, binding_sources()) or not os.path.exists(BUILT_FOR):
        return False
    with open(BUILT_FOR) as f:
        return f.read() == installed_torch()


def binding_sources():
    return [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "bpt.h")]


def _newer(built: str, sources) -> bool:
    return os.path.exists(built) and all(os.path.getmtime(p) <= os.path.getmtime(built) for p in sources)


def build_binding() -> str:
    """The g++ on PATH, as nvcc takes for the library (a compiler that links its own static libstdc++ would put a
    second one, with locales of its own, beside torch's), against the installed torch; finds libbpt.so beside itself."""
    import torch

    home = os.path.dirname(torch.__file__)
    lib = os.path.join(home, "lib")
    include = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), sysconfig.get_paths()["include"]]
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           *[f"-isystem{p}" for p in include], "-o", tmp,
           os.path.join(CSRC, "binding.cpp"), "-L", PKG, "-l:libbpt.so", "-Wl,-rpath,$ORIGIN", "-L", lib, "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", f"-Wl,-rpath,{lib}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed ({res.returncode}):\n{res.stdout + res.stderr}")
    os.replace(tmp, BINDING)
    with open(BUILT_FOR, "w") as f:
        f.write(installed_torch())
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _newer(LIB, sources()):
        build_library(verbose)
    if installed_torch() is None:
        print("torch is not installed: the C library was built, the Python binding was not", file=sys.stderr)
    elif force or not binding_up_to_date():
        build_binding()
    return LIB


def build_library(verbose: bool = False) -> str:
    cu = [p for p in sources() if p.endswith(".cu")]
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-o", tmp, *cu]
    res = subprocess.run(cmd, capture_output=True, text=True)
    log = res.stdout + res.stderr
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{log}")
    os.replace(tmp, LIB)
    with open(os.path.join(PKG, "build.log"), "w") as f:
        f.write(" ".join(cmd) + "\n" + log)
    if verbose:
        print(log)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
