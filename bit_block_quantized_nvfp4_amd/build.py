"""Build libmoe_nvfp4.so (HIP, gfx950) in-tree with hipcc, and _binding.so.

Each ``csrc/*.hip`` file is compiled to an object under ``_build/`` in
parallel, then linked into ``libmoe_nvfp4.so`` next to this file.  Every HIP
file is compiled with packed-FP32 instructions disabled.  ``csrc/binding.cpp``
is host code only: a Python module beside it that checks and passes on torch
tensors.  The library stands by itself: it is in place before the module is
begun, and where torch is missing the module is left out.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_nvfp4.so")
BINDING = os.path.join(HERE, "_binding.so")
ARCH = "gfx950"

HIP_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Wall", "-Wno-unused-function",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found: the MoE library needs ROCm's hipcc")


def cxx() -> str:
    """The host compiler of the Python module: CXX, g++, or ROCm's own clang++."""
    for c in (os.environ.get("CXX"), "g++", os.path.join(os.path.dirname(hipcc()), "amdclang++")):
        if c and shutil.which(c):
            return c
    raise RuntimeError("no host C++ compiler found for the Python module (the library itself is built)")


def binding_command(out: str) -> list:
    import torch
    from torch.utils import cpp_extension

    inc = [*cpp_extension.include_paths(), os.path.join(os.path.dirname(os.path.dirname(hipcc())), "include"),
           sysconfig.get_paths()["include"]]
    return [cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f for p in inc for f in ("-isystem", p)], os.path.join(CSRC, "binding.cpp"), "-o", out,
            "-L" + cpp_extension.TORCH_LIB_PATH, "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python",
            "-L" + HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]


def build_library(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = hipcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    procs = []
    objs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s) + ".o")
        objs.append(o)
        cmd = [cc, *HIP_FLAGS, "-c", s, "-o", o]
        if verbose:
            print(" ".join(cmd))
        procs.append((s, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for s, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        # the host pass does not know the packed-fp32 feature; that note is harmless
        lines = [ln for ln in text.splitlines() if "packed-fp32-ops" not in ln]
        if p.returncode != 0:
            failed.append((s, "\n".join(lines)))
        elif verbose and lines:
            print("\n".join(lines))
    if failed:
        msg = "\n\n".join(f"== {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"HIP compile failed:\n{msg}")
    tmp = LIB + ".tmp"
    cmd = [cc, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)
    return LIB


def build_binding() -> str:
    tmp = BINDING + ".tmp"
    r = subprocess.run(binding_command(tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError(f"binding compile failed ({LIB} is built):\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, BINDING)
    return BINDING


def build(verbose: bool = False) -> str:
    build_library(verbose)
    if importlib.util.find_spec("torch") is None:
        print("torch is not installed: the C library alone is built, without the Python module", file=sys.stderr)
    else:
        build_binding()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
