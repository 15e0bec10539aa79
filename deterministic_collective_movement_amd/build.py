"""Build librog.so (the C-ABI library) in-tree for gfx950.

``build_library()`` compiles the host planners and the HIP kernels (gathers,
rank-ordered sums, token log probabilities, the policy loss and the policy
head's products) with hipcc for
gfx950, then links ``deterministic_collective_movement_amd/librog.so``.
Intermediate objects go to ``_build/`` at the repository root.
``python -m deterministic_collective_movement_amd.build`` does the same.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "librog.so")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
ARCH = "gfx950"

HOST_SOURCES = ["rog_plan.cpp", "rog_head_plan.cpp", "rog_linear_plan.cpp"]
HIP_SOURCES = ["rog_kernels.hip", "rog_reduce.hip", "rog_logprob.hip", "rog_logprob_grad.hip", "rog_policy.hip",
               "rog_linear_score.hip", "rog_linear_grad.hip", "rog_linear_i8.hip"]

# Device code: gfx950 only; packed-FP32 instructions disabled.
HIP_FLAGS = ["-O3", "-std=c++17", "-fPIC", "-Wall", "-Wextra", "-Werror",
             "--offload-arch=" + ARCH,
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-Wno-unused-command-line-argument"]
# Host planner: compiled as HIP source too (it shares the payload-cut helper
# with the kernels), but it holds host code only.
HOST_FLAGS = ["-x", "hip", "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wextra", "-Werror",
              "--offload-arch=" + ARCH, "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
              "-Wno-unused-command-line-argument"]


BINDING_SOURCE = "rog_binding.cpp"
BINDING_PATH = os.path.join(PKG, "_rog_binding.so")


def _run(cmd):
    subprocess.check_call(cmd)


def build_library(out: str = LIB_PATH, defines=(), build_dir: str = BUILD_DIR) -> str:
    """Compile and link librog.so; ``defines`` (e.g. ["ROG_VEC_UNROLL=8"]) go to both compilers."""
    hipcc = shutil.which("hipcc") or os.path.join(ROCM, "bin", "hipcc")
    os.makedirs(build_dir, exist_ok=True)
    inc = ["-I", INCLUDE, "-I", CSRC, "-I", os.path.join(ROCM, "include")]
    dflags = ["-D" + d for d in defines]
    # independent translation units, compiled side by side
    jobs, objs = [], []
    for src in HOST_SOURCES + HIP_SOURCES:
        obj = os.path.join(build_dir, os.path.splitext(src)[0] + ".o")
        flags = HOST_FLAGS if src in HOST_SOURCES else HIP_FLAGS
        objs.append(obj)
        jobs.append([hipcc] + flags + dflags + inc + ["-c", os.path.join(CSRC, src), "-o", obj])
    with ThreadPoolExecutor(max_workers=8) as pool:
        list(pool.map(_run, jobs))
    tmp = out + ".tmp%d" % os.getpid()
    _run([hipcc, "-shared", "-fPIC", "--offload-arch=" + ARCH] + objs +
         ["-Wl,-soname,librog.so", "-Wl,-rpath," + os.path.join(ROCM, "lib"), "-Wl,--no-undefined", "-o", tmp])
    os.replace(tmp, out)
    return out


def build_binding(out: str = BINDING_PATH) -> str:
    """Compile and link _rog_binding.so, the CPython module beside librog.so (host
    code only; against the installed torch's headers and libraries)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    inc = [f for d in [INCLUDE, os.path.join(ROCM, "include"), sysconfig.get_paths()["include"]] + cpp_extension.include_paths()
           for f in ("-isystem", d)]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = out + ".tmp%d" % os.getpid()
    _run([shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wextra", "-Werror",
          "-D__HIP_PLATFORM_AMD__", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI] + inc +
         [os.path.join(CSRC, BINDING_SOURCE), "-o", tmp, "-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cpu", "-lc10"])
    os.replace(tmp, out)
    return out


def build_all() -> None:
    """Everything the package loads."""
    with ThreadPoolExecutor(max_workers=1) as pool:
        binding = pool.submit(build_binding)
        build_library()
        binding.result()


if __name__ == "__main__":
    if sys.argv[1:]:
        print(build_library(defines=sys.argv[1:]))
    else:
        build_all()
        print(LIB_PATH)
        print(BINDING_PATH)
