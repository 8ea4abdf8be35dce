"""Build the gfx950 shared library libmoe_mi355x.so, and the binding's extension
module _calls, in-tree with hipcc.

    python -m sigmoid_top_routing_router_amd.build

Every source under csrc/ is compiled to an object (in parallel) and linked
into one shared library next to this file.  The build always recompiles.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor
from importlib.machinery import EXTENSION_SUFFIXES

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_mi355x.so")
BINDING = os.path.join(HERE, "_calls" + EXTENSION_SUFFIXES[0])
ARCH = "gfx950"

HIPFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build the library)")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".hip", ".cpp")))


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [hipcc(), *HIPFLAGS, "-I", os.path.join(HERE, "..", "include"), "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def build_binding(verbose: bool = False) -> str:
    """The extension module of the Python binding: host code against the installed
    torch."""
    import sysconfig

    from torch.utils.cpp_extension import include_paths, library_paths

    from ._lib import built_for
    out = BINDING
    cmd = [hipcc(), "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", f'-DMOE_BUILT_FOR="{built_for()}"',
           "-I", "/opt/rocm/include",
           *(f for p in include_paths() for f in ("-isystem", p)),
           "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "binding", "calls.cpp"), "-o", out + ".tmp",
           *(f for p in library_paths() for f in ("-L", p)),
           "-lc10", "-lc10_hip", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"binding build failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(out + ".tmp", out)
    if verbose:
        print(f"built {out}")
    return out


PROBES = os.path.join(HERE, "..", "tests", "probes")


def build_probes(verbose: bool = False):
    """Test probes: small stand-alone HIP programs that measure a property of
    the hardware that a parity tolerance rests on (tests/probes/*.hip ->
    executables next to them)."""
    out = []
    for f in sorted(os.listdir(PROBES)) if os.path.isdir(PROBES) else []:
        if not f.endswith(".hip"):
            continue
        src = os.path.join(PROBES, f)
        exe = src[:-4]
        cmd = [hipcc(), *HIPFLAGS, src, "-o", exe]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"probe build failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        out.append(exe)
        if verbose:
            print(f"built {exe}")
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = sources()
    with ThreadPoolExecutor(max(1, min(8, len(srcs) + 1))) as ex:
        binding = ex.submit(build_binding, verbose)
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print(f"built {LIB}")
    # the library needs hipcc alone, the binding works without its module: a host without
    # torch's or Python's headers has the library all the same
    try:
        binding.result()
    except Exception as e:
        if os.path.exists(BINDING):  # of an earlier build
            os.remove(BINDING)
        warnings.warn(f"built without the binding's extension module, small calls take twice "
                      f"the time on the host: {e}")
    build_probes(verbose)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
