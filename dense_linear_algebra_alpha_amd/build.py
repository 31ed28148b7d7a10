"""Builds libxtvxy.so (the fused kernels and the C ABI) for gfx950 with hipcc, and
_tensors.so (a small host-only Python extension of the torch helpers) with g++.
The library does not need the extension: without torch or g++ it is built alone.

Objects go to _build/ next to this file and the shared libraries next to this
file, so it travels with the source tree. Usage: ``python -m
dense_linear_algebra_alpha_amd.build`` or ``build()`` from Python.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libxtvxy.so")
TENSORS_PATH = os.path.join(HERE, "_tensors.so")  # Python extension: checked addresses of tensor lists
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
HIPCC = os.path.join(ROCM, "bin", "hipcc")
ARCH = "gfx950"

SOURCES = ["api.cpp", "model.cpp", "unfused.cpp", "logreg.cpp", "tune.cpp", "csr_analysis.cpp", "dense.hip", "csr.hip",
           "csr_waves.hip", "csr_rows.hip", "csr_bins.hip",
           "aggregate.hip", "logreg.hip", "probe.hip", "noalloc.hip",
           "linear.cpp", "linear_tile.hip", "linear_ring.hip", "linear_few.hip", "adamw.cpp", "adamw.hip",
           "norm.cpp", "norm.hip", "embedding.cpp", "embedding.hip",
           "loss.cpp", "loss.hip"]
TENSORS_SOURCE = "tensor_list.cpp"
HEADERS = ["internal.h", "device_util.h", "csr_common.h", "linear.h", "linear_util.h", "adamw.h", "matrix.h", "norm.h", "embedding.h",
           "loss.h", "linear_plan.h", "linear_ring.h"]

COMMON_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
    "-I" + INCLUDE, "-I" + CSRC,
]
# Device code: gfx950 only; hardware float atomics; packed-fp32 instructions off.
DEVICE_FLAGS = [
    "--offload-arch=" + ARCH, "-munsafe-fp-atomics",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(src: str) -> str:
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD_DIR, src + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC] + COMMON_FLAGS + DEVICE_FLAGS + lang + ["-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature; drop that line
    noise = "is not a recognized feature for this target"
    msgs = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed on %s:\n%s" % (src, msgs))
    if msgs.strip():
        print(msgs, file=sys.stderr)
    return obj


def _extension_lacks() -> str:
    """What the extension module cannot be built without and is not there, or an empty string."""
    if importlib.util.find_spec("torch") is None:
        return "torch"
    return "" if shutil.which("g++") else "g++"


def _build_tensors() -> None:
    """The host-only extension module, against the headers of the installed torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    tmp = TENSORS_PATH + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-DUSE_ROCM",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)]
    cmd += ["-isystem" + d for d in cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]]
    # torch's libraries are found by name among those that the process has loaded by importing torch
    cmd += [os.path.join(CSRC, TENSORS_SOURCE), "-o", tmp, "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
            "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on %s:\n%s%s" % (TENSORS_SOURCE, r.stdout, r.stderr))
    os.replace(tmp, TENSORS_PATH)


def build(verbose: bool = False) -> str:
    """Compile every source, link libxtvxy.so and build the extension module; returns the library path. The
    library is there also where the extension's build fails."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 1)) as ex:
        lacks = _extension_lacks()
        tensors = None if lacks else ex.submit(_build_tensors)
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs + [
        "-L" + os.path.join(ROCM, "lib"), "-lrocblas", "-lrocsparse", "-Wl,-rpath," + os.path.join(ROCM, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB_PATH)
    if verbose:
        print("built", LIB_PATH)
    if lacks:
        print("_tensors.so is not built without %s: the torch helpers work, with more host time a call" % lacks,
              file=sys.stderr)
    else:
        tensors.result()
    return LIB_PATH


def sources_newer_than_library() -> bool:
    extension = not _extension_lacks()
    if not os.path.exists(LIB_PATH) or (extension and not os.path.exists(TENSORS_PATH)):
        return True
    t = os.path.getmtime(LIB_PATH)
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "xtvxy.h")]
    return any(os.path.getmtime(f) > t for f in files) or (
        extension and os.path.getmtime(os.path.join(CSRC, TENSORS_SOURCE)) > os.path.getmtime(TENSORS_PATH))


if __name__ == "__main__":
    build(verbose=True)
