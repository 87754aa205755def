"""Build the gfx950 HIP library libqmv.so in-tree (hipcc, one object per
kernel-instance unit, compiled in parallel, then linked), and the torch binding
qmv_ops_py.so beside it (g++).  The library needs hipcc alone: without torch, g++ or
Python's headers it is built without the binding, and so are the C ABI's users served."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libqmv.so")
PY = os.path.join(LIBDIR, "qmv_ops_py.so")
ROCM = "/opt/rocm"
HIPCC = os.environ.get("HIPCC", os.path.join(ROCM, "bin", "hipcc"))

# -ffp-contract=off: every fused multiply-add in the kernels is written out
# explicitly, so no instance can fuse differently from another.  Packed fp32
# instructions are turned off for all HIP code.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-I", os.path.join(ROOT, "include"), "-I", CSRC]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", src, "-o", obj]
    _run(cmd, f"hipcc failed on {src}")
    return obj


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(what)


def _binding_lacks() -> str | None:
    """What the binding's build would need and is not here."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    if shutil.which("g++") is None:
        return "g++"
    header = os.path.join(sysconfig.get_paths()["include"], "Python.h")
    return None if os.path.exists(header) else header


def _compile_binding() -> str:
    import torch
    obj = os.path.join(BUILD, "ops_py.o")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-DUSE_ROCM", "-D__HIP_PLATFORM_AMD__=1",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", os.path.join(ROOT, "include"),
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", f"{ROCM}/include",
          "-isystem", sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "ops_py.cpp"), "-o", obj],
         "g++ failed on ops_py.cpp")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    _run(["g++", "-shared", "-o", PY + ".tmp", obj, "-L", LIBDIR, "-lqmv", "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
          "-lc10", "-ltorch_cpu", "-ltorch_python", "-lc10_hip", "-ltorch_hip", "-Wl,-rpath,$ORIGIN"],
         "link of qmv_ops_py.so failed")
    os.replace(PY + ".tmp", PY)


def build(jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    jobs = jobs or min(8, os.cpu_count() or 1)
    lacks = _binding_lacks()
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        binding = None if lacks else ex.submit(_compile_binding)
        objs = list(ex.map(_compile, sources()))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    _run(cmd, "link of libqmv.so failed")
    os.replace(tmp, LIB)
    if lacks:
        sys.stderr.write(f"{os.path.basename(PY)} is not built (no {lacks}): the calls of ops.py need it\n")
    else:
        _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build())
