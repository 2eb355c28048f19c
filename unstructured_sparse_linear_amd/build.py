"""Build libspops.so (the HIP kernels and the C ABI) for gfx950 with hipcc, and
_marshal.so (the compiled part of the Python binding) with the host compiler.

Each .hip source under csrc/ is compiled to an object in parallel, then the
objects are linked into libspops.so next to this file.  Always rebuilds.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build", "spops")
LIB = os.path.join(HERE, "libspops.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
CEILINGS_LIB = os.path.join(HERE, "libspops_ceilings.so")
ARCH = os.environ.get("SPOPS_OFFLOAD_ARCH", "gfx950")

CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall",
    "-fno-gpu-flush-denormals-to-zero",
    # packed fp32 VALU forms stay off: ordinary fp32 code is emitted instead
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def _hipcc() -> str:
    h = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(h):
        raise RuntimeError("hipcc not found; the HIP library cannot be built")
    return h


def _compile(src: str) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    cmd = [_hipcc(), *CFLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _run(cmd: list, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stderr}")


def _compile_marshal() -> str:
    """csrc/marshal.cpp against the installed torch's headers; host code only."""
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(OBJDIR, "marshal.cpp.o")
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(_hipcc())))
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
          "-I", INCLUDE, "-isystem", inc,
          "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", os.path.join(rocm, "include"),
          "-isystem", sysconfig.get_paths()["include"],
          "-c", os.path.join(CSRC, "marshal.cpp"), "-o", obj], "g++ for marshal.cpp")
    return obj


def _link_marshal(obj: str) -> str:
    import torch
    tlib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL + ".tmp"
    _run(["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libspops.so", "-Wl,-rpath,$ORIGIN",
          "-L", tlib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip",
          f"-Wl,-rpath,{tlib}"], "link of _marshal.so")
    os.replace(tmp, MARSHAL)
    return MARSHAL


def build(jobs: int | None = None, verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.hip")))
    jobs = jobs or min(len(srcs), os.cpu_count() or 4, 16)
    with cf.ThreadPoolExecutor(jobs) as ex:
        marshal = ex.submit(_compile_marshal)
        objs = list(ex.map(_compile, srcs))
        marshal_obj = marshal.result()
    tmp = LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_marshal(marshal_obj)
    if verbose:
        print(f"built {LIB}", file=sys.stderr)
        print(f"built {MARSHAL}", file=sys.stderr)
    build_ceilings(verbose)
    return LIB


def build_ceilings(verbose: bool = False) -> str:
    """The benchmark's measurement kernels (gather rates), a library of their
    own that libspops does not link."""
    src = os.path.join(HERE, "ceilings", "ceilings.hip")
    obj = _compile(src)
    tmp = CEILINGS_LIB + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, CEILINGS_LIB)
    if verbose:
        print(f"built {CEILINGS_LIB}", file=sys.stderr)
    return CEILINGS_LIB


if __name__ == "__main__":
    build(verbose=True)
