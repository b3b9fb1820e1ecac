"""Build the gfx950 HIP library ``libconv2d_gi.so`` in-tree with hipcc.

Usage: ``python -m conv2d_backward_amd.build`` (or ``build()`` from Python).
Each source compiles to an object under ``_build/`` at the repository root,
in parallel; the objects link into ``conv2d_backward_amd/libconv2d_gi.so``.
Beside it ``_sequence.so`` is built, the extension module behind sequence.py, which
needs torch and g++; without torch only the library is built.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libconv2d_gi.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = [
    "api.cpp",
    "kernels_generic.hip",
    "kernels_halo_f32.hip",
    "kernels_halo_bf16.hip",
    "kernels_img16.hip",
    "kernels_stem_f32.hip",
    "kernels_col2im_f32.hip",
    "kernels_gw_f32.hip",
    "kernels_fwd_f32.hip",
    "noalloc.hip",
    "kernels_causal_conv.hip",
    "kernels_state_scan.hip",
    "kernels_state_scan_bwd.hip",
    "kernels_block_norm.hip",
    "seq_api.cpp",
    "kernels_peak.hip",
]

COMMON = ["-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall", "-Werror",
          "--offload-arch=" + ARCH, "-I", INCLUDE, "-I", CSRC]
# Device code: gfx950 only; packed fp32 instructions are switched off.
DEVICE = ["-x", "hip", "--offload-arch=" + ARCH,
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Wno-unused-command-line-argument"]


# The extension module behind sequence.py: host code against torch's C++ API.
BINDING = "seq_binding.cpp"
BINDING_PATH = os.path.join(PKG, "_sequence.so")


def _build_binding() -> str | None:
    import sysconfig

    try:
        import torch
        from torch.utils import cpp_extension
    except ImportError as e:
        sys.stderr.write("%s is not built: no torch (%s)\n" % (os.path.basename(BINDING_PATH), e))
        return None

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", "-Wall", "-Werror", "-Wno-sign-compare",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
    for d in cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]:
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, BINDING), "-o", tmp, "-L", lib, "-Wl,-rpath," + lib,
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s\n%s" % (BINDING, " ".join(cmd), r.stderr))
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def _compile(src: str) -> str:
    path = os.path.join(CSRC, src)
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC] + COMMON + (DEVICE if src.endswith(".hip") else []) + ["-c", path, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the gfx950 feature name; that warning is noise.
    err = "\n".join(l for l in r.stderr.splitlines()
                    if "is not a recognized feature for this target" not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), err))
    if err.strip():
        sys.stderr.write(err + "\n")
    return obj


def build(verbose: bool = False) -> str:
    """Compile every source for gfx950, link the shared library and build its torch binding
    (always rebuilds)."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(_compile, SOURCES))
        # The library is whole before what becomes of its binding counts.
        tmp = LIB_PATH + ".tmp%d" % os.getpid()
        cmd = [HIPCC, "-shared", "-fPIC", "--offload-arch=" + ARCH, "-o", tmp] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
        os.replace(tmp, LIB_PATH)
        binding.result()
    if verbose:
        print("built", LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    build(verbose=True)
