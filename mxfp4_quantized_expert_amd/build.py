"""Build libmxfp4moe.so (gfx950 only) from csrc/*.hip with hipcc, in-tree.

Usage: python -m mxfp4_quantized_expert_amd.build
"""

from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmxfp4moe.so")
HOST_CALLS = os.path.join(PKG, "_host_calls.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    "-Wno-unused-result",
    # keep the compiler from forming packed-fp32 vector ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{os.path.join(ROOT, 'include')}",
]


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    msg = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{msg}")
    if msg.strip():
        print(msg, file=sys.stderr)
    return obj


def _build_host_calls() -> bool:
    """csrc/host_calls.cpp, the Python module of the short host path, beside the library it calls.  It needs
    g++ and the headers of Python and torch; where it cannot be built, none is left (one of an earlier
    library would call this one), and the binding calls through ctypes."""
    try:
        import sysconfig

        import torch

        torch_dir = os.path.dirname(torch.__file__)
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               "-isystem", os.path.join(torch_dir, "include"), "-isystem", sysconfig.get_paths()["include"],
               os.path.join(CSRC, "host_calls.cpp"), "-o", HOST_CALLS + ".tmp",
               f"-L{PKG}", "-lmxfp4moe", "-Wl,-rpath,$ORIGIN",
               f"-L{os.path.join(torch_dir, 'lib')}", "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = "" if r.returncode == 0 else r.stdout + r.stderr or f"{cmd[0]} ended with {r.returncode}"
    except (ImportError, OSError) as e:
        why = str(e)
    if why:
        if os.path.exists(HOST_CALLS):
            os.remove(HOST_CALLS)
        print(f"{HOST_CALLS} was not built, calls take the longer way through ctypes:\n{why}", file=sys.stderr)
        return False
    os.replace(HOST_CALLS + ".tmp", HOST_CALLS)
    return True


def build(verbose: bool = True) -> str:
    """Compile every csrc/*.hip for gfx950 and link libmxfp4moe.so next to this file, then, where that
    can be done, the Python module that calls it."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(_compile, srcs))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
    os.replace(tmp, LIB)
    _build_host_calls()
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
