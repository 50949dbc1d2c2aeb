"""Build libfp8w8a8.so (and bench.py's libhbmprobe.so) in-tree with hipcc
for gfx950, and the binding's _tensor_args extension with the host compiler.

    python -m fp8_w8a8_block_amd.build        # or fp8_w8a8_block_amd.build.build()

Every source is compiled to an object (in parallel), then linked into the
package directory.  Flags: -O3, no fast-math, no fp contraction (fused
multiply-adds are written out where they are meant), packed-fp32 VALU ops
switched off.
"""

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfp8w8a8.so")
SOURCES = ["abi.hip", "quant_kernels.hip", "gemm_kernels.hip", "kv_kernels.hip",
           "attention_abi.hip", "slot_kernels.hip", "rope_kernels.hip", "attention_kernels.hip",
           "step_abi.hip", "norm_kernels.hip", "int4_kernels.hip", "logprob_kernels.hip"]
PROBE_SOURCE = "hbm_probe.hip"                 # bench.py's HBM and matrix-unit references
PROBE_LIB = os.path.join(PKG, "libhbmprobe.so")
ARGS_SOURCE = "tensor_args.cpp"                # the binding's reader of tensor arguments
ARGS_LIB = os.path.join(PKG, "_tensor_args.so")
ARCH = "gfx950"


def hipcc():
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found; ROCm is required to build the library")
    return path


def common_flags():
    return [
        "-O3", f"--offload-arch={ARCH}", "-std=c++17", "-fPIC",
        "-ffp-contract=off", "-fno-fast-math",
        "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
        "-Wall", "-Wno-unused-function", "-Wno-unused-command-line-argument",
        "-I", INCLUDE, "-I", CSRC,
    ]


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [hipcc()] + common_flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    noise = [l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l and l.strip()]
    if verbose and noise:
        print("\n".join(noise), flush=True)
    return obj


def _build_args(verbose):
    """The extension module: host code against torch's own headers."""
    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    tmp = ARGS_LIB + ".tmp"
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
           os.path.join(CSRC, ARGS_SOURCE), "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch_cpu",
           "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {ARGS_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, ARGS_LIB)


def build(verbose=False):
    """Compile every HIP source for gfx950 and link the shared library."""
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs + [
        "-Wl,-rpath,/opt/rocm/lib"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    # bench.py's HBM read and matrix-unit references, a library of their own
    probe = _compile(PROBE_SOURCE, verbose)
    tmp = PROBE_LIB + ".tmp"
    r = subprocess.run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, probe,
                        "-Wl,-rpath,/opt/rocm/lib"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, PROBE_LIB)
    _build_args(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
