"""Build the HIP library libglu_gemv.so for gfx950, in place.

Each ``csrc/*.hip`` compiles to an object in parallel, then they link into a
shared library next to this file; ``csrc/glu_torch.cpp`` becomes the extension
module ``_fast``.  Flags: gfx950 only, -O3, no fast math, no
FP contraction beyond the explicit fmaf calls, packed-FP32 instructions
disabled (the compiler forms them from scalar float code on its own), code
object v5.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIBRARY = os.path.join(HERE, "libglu_gemv.so")
BINDING = os.path.join(HERE, "_fast.so")  # host code only: torch tensors to the C ABI (csrc/glu_torch.cpp)
ROOT = os.path.dirname(HERE)
INCLUDE = os.path.join(ROOT, "include")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

HIP_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-mcode-object-version=5",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
    f"-I{INCLUDE}",
]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC, *HIP_FLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    noise = "unknown target feature"  # the host pass does not know the device-only feature
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l and "packed-fp32" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{err}")
    if err.strip() and verbose:
        print(err, file=sys.stderr)
    return obj


def build_binding(verbose: bool = False) -> str:
    """Compile the torch binding _fast.so (host C++ against torch's headers); returns its path."""
    import torch
    from torch.utils import cpp_extension

    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f for p in cpp_extension.include_paths() for f in ("-isystem", p)], "-isystem",
           os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"), "-I" + sysconfig.get_paths()["include"],
           os.path.join(CSRC, "glu_torch.cpp"), "-o", tmp, "-L" + cpp_extension.TORCH_LIB_PATH, "-lc10", "-lc10_hip",
           "-ltorch_cpu", "-ltorch_hip", "-ltorch_python", "-Wl,-rpath," + cpp_extension.TORCH_LIB_PATH]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on glu_torch.cpp:\n{res.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def build(verbose: bool = False, jobs: int = 8) -> str:
    """Compile every HIP source, link libglu_gemv.so and compile the torch binding; returns the library's path.

    The library is linked whatever becomes of the binding, whose failure is raised after it: callers of the C ABI need
    no torch headers.
    """
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(jobs, len(srcs)))) as ex:
        binding = ex.submit(build_binding, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIBRARY + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIBRARY)
    binding.result()
    return LIBRARY


if __name__ == "__main__":
    print(build(verbose=True))
