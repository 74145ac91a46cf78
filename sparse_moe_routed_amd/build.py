"""Compile the HIP kernels and the C-ABI layer into ``libmoe.so`` (gfx950),
and the Python binding of the calls around the layer into ``_block.so`` (host
code against torch's headers).  The library needs hipcc only: without g++,
Python's headers or torch it is built alone.

Run ``python -m sparse_moe_routed_amd.build`` (or ``__graft_entry__.build()``).
It always recompiles; objects go to ``_build/`` at the repository root.
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe.so")
BINDING = os.path.join(PKG, "_block.so")
ARCH = "gfx950"

# packed-fp32 instructions are disabled for all device code; MFMA results go
# to VGPRs (the low-bit kernels scale each MFMA result with VALU FMAs, and the
# default AGPR destinations cost one v_accvgpr_read per element)
HIPCC_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-result", "-Wno-pass-failed",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "--amdgpu-mfma-vgpr-form",
    "-I", os.path.join(ROOT, "include"),
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith(".hip") or f.endswith(".cpp"))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [hipcc(), *HIPCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in r.stderr.splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{err}")
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed: {' '.join(cmd)}\n{r.stderr}")


def _binding_lacks() -> str | None:
    """What is not there to build the binding with, if anything."""
    if not shutil.which("g++"):
        return "g++"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    try:
        import torch
    except ImportError:
        return "torch"
    header = os.path.join(os.path.dirname(torch.__file__), "include", "torch", "csrc", "autograd",
                          "python_variable.h")
    return None if os.path.exists(header) else "torch's headers"


def _compile_binding() -> str:
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    obj = os.path.join(BUILD, "block_binding.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
          "-D__HIP_PLATFORM_AMD__", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-I", os.path.join(ROOT, "include"), "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(rocm, "include"),
          "-isystem", sysconfig.get_paths()["include"],
          "-c", os.path.join(PKG, "binding", "block_binding.cpp"), "-o", obj], "binding compile")
    return obj


def _link_binding(obj: str, lib: str, out: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    # libmoe.so (its soname) beside it; torch and the HIP runtime are loaded by torch
    _run(["g++", "-shared", "-o", out, obj, lib, "-Wl,-rpath,$ORIGIN", "-L", libs,
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,--as-needed"], "binding link")


def build(verbose: bool = True) -> str:
    """Both files are replaced once both are linked: a build that fails leaves
    the older pair, and a library is never left beside a binding of another."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    lacks = _binding_lacks()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        binding = None if lacks else ex.submit(_compile_binding)
        objs = list(ex.map(_compile, srcs))
    lib, block = LIB + ".tmp", BINDING + ".tmp"
    _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-Wl,-soname,libmoe.so", "-o", lib, *objs],
         "link")
    if binding:
        _link_binding(binding.result(), lib, block)
    if os.path.exists(BINDING):
        os.remove(BINDING)
    os.replace(lib, LIB)
    if binding:
        os.replace(block, BINDING)
    else:
        sys.stderr.write(f"{os.path.basename(BINDING)} was not built, {lacks} is missing: the calls around "
                         "the layer have no Python binding\n")
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
