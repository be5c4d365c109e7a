"""Build libqgemm.so in-tree with hipcc for gfx950 (CDNA4 / MI355X).

The library's HIP sources under ``csrc/`` are compiled to objects in
parallel and linked into ``conv_qgemm_amd/libqgemm.so``; the benchmark's
calibration kernels (``csrc/calib.hip``) go to their own
``conv_qgemm_amd/libqgcalib.so``; the Python callables of the decoding
step's entry points (host code only, for the torch that it is built with) to
``conv_qgemm_amd/_qcall.so``.  Objects go to ``_build/`` at the repository
root.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "_build", "qgemm")
LIB = os.path.join(PKG, "libqgemm.so")
CALIB_LIB = os.path.join(PKG, "libqgcalib.so")
CALIB_SOURCES = ["calib.hip"]
# the benchmark's comparison with AMD's hipBLASLt int8 GEMM (its own library,
# so that libqgemm.so does not depend on hipBLASLt)
VENDOR_LIB = os.path.join(PKG, "libqgvendor.so")
VENDOR_SOURCES = ["vendor_hipblaslt.cpp"]
SOURCES = ["api.cpp", "k_tile_gemm.hip", "k_gemm_dma.hip", "k_gemm_dma_dequant.hip", "k_skinny_w4a8.hip", "k_conv_halo.hip", "k_dwconv.hip",
           "k_quant.hip", "k_zp.hip", "k_dequant_gemm.hip", "k_kv_cache.hip", "k_attn_kv8.hip"]

# Python callables of some entry points (a module for this interpreter)
CALL_LIB = os.path.join(PKG, "_qcall.so")
CALL_SOURCE = "pycall.cpp"

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++20", "-fPIC", "-Wall",
    "-mcode-object-version=5",
    # no packed-fp32 instruction selection
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{os.path.join(ROOT, 'include')}",
]
# Per-source additions.  The attention kernels make no NaN from the finite
# values that they take (masked scores are -infinity and never meet a factor of
# 0, scales of 0 are held above it: attn_weights.hpp): without that promise
# every maximum first re-rounds its operands.
# The large-GEMM ring keeps its 256 accumulators of
# 16x16 MFMA tiles in place only when the pre-RA machine scheduler is off:
# with it, the compiler reorders the loop's MFMAs so that about half of them
# write a different register quad than they read, and every K stage then
# pays 130-230 accumulator copies (measured in the generated code, and in the
# kernel: the matrix pipe busy 54% instead of 65%).  The loop's source order
# is already the intended schedule.
SRC_FLAGS = {
    "k_gemm_dma.hip": ["-mllvm", "-enable-misched=0"],
    "k_gemm_dma_dequant.hip": ["-mllvm", "-enable-misched=0"],
    "k_attn_kv8.hip": ["-fno-honor-nans"],
}


def flags_for(src: str):
    """Compiler flags of one source file under csrc/."""
    return [*CFLAGS, *SRC_FLAGS.get(os.path.basename(src), [])]


def _compile(src: str) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    cmd = [HIPCC, *flags_for(src), "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def _link(objs, lib, verbose, libs=()):
    tmp = lib + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp,
           "-Wl,-rpath,/opt/rocm/lib", *libs]
    subprocess.run(cmd, check=True, capture_output=not verbose)
    os.replace(tmp, lib)
    if verbose:
        print(f"built {lib}", file=sys.stderr)


def _build_call(verbose):
    # only paths and the ABI flag come from torch here, not its GPU side
    import torch
    base = os.path.join(os.path.dirname(torch.__file__))
    inc = os.path.join(base, "include")
    tmp = CALL_LIB + ".tmp"
    cmd = ["g++", "-O2", "-std=c++20", "-fPIC", "-Wall", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{os.path.join(ROOT, 'include')}", "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], os.path.join(CSRC, CALL_SOURCE),
           f"-L{os.path.join(base, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALL_SOURCE}:\n{r.stderr}")
    os.replace(tmp, CALL_LIB)
    if verbose:
        print(f"built {CALL_LIB}", file=sys.stderr)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = SOURCES + CALIB_SOURCES + VENDOR_SOURCES
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), 8)) as ex:
        call = ex.submit(_build_call, verbose)
        objs = list(ex.map(_compile, srcs))
    n, c = len(SOURCES), len(CALIB_SOURCES)
    _link(objs[:n], LIB, verbose)
    _link(objs[n:n + c], CALIB_LIB, verbose)
    _link(objs[n + c:], VENDOR_LIB, verbose, libs=["-L/opt/rocm/lib", "-lhipblaslt"])
    call.result()  # a failure there leaves the libraries linked
    return LIB


if __name__ == "__main__":
    build(verbose=True)
