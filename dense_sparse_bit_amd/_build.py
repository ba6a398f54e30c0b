"""Build libmq.so (the HIP library) in-tree with hipcc for gfx950, and _binding.so (the
extension module that calls it) with g++.

    python dense_sparse_bit_amd/_build.py

A standalone script (it imports nothing from the package, whose import needs the
built library). Cross-compiles without a GPU. Objects go to
dense_sparse_bit_amd/_build/, the libraries to dense_sparse_bit_amd/.
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmq.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = [
    f"--offload-arch={ARCH}", "-O3", "-fPIC", "-std=c++17", "-Wall",
    # packed fp32 instructions stay off: plain fp32 code only
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # IEEE behaviour the bit-exact steps rely on
    "-fhip-fp32-correctly-rounded-divide-sqrt", "-fno-gpu-flush-denormals-to-zero",
    "-fno-fast-math",
]
# per-source extra flags: the preparation kernels must not contract a*b+c
SOURCES = {
    "prep.hip": ["-ffp-contract=off"],
    "gemm.hip": [],
    "api.hip": ["-ffp-contract=off"],
    "mx_quant.hip": [],
    "mx_gemm.hip": [],
    "route.hip": ["-ffp-contract=off"],
    "api_mx.hip": [],
}


def _compile(name: str, flags: list) -> str:
    src = os.path.join(CSRC, name)
    out = os.path.join(OBJ, name.replace(".hip", ".o"))
    cmd = [HIPCC, *COMMON, *flags, "-c", src, "-o", out]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {name}:\n{r.stderr}")
    return out


def _binding() -> str:
    """The extension module: host code against torch's headers and libmq.so. It holds the
    versions that it is built for, and does not load with others."""
    spec = importlib.util.find_spec("torch")              # found, not imported
    torch = os.path.dirname(spec.origin)
    spec = importlib.util.spec_from_file_location("_torch_version", os.path.join(torch, "version.py"))
    version = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(version)
    out = os.path.join(PKG, "_binding.so")
    cmd = ["g++", "-O2", "-fPIC", "-shared", "-std=c++17", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f'-DMQ_TORCH_VERSION="{version.__version__}"',
           "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"), "-o", out + ".tmp",
           f"-L{torch}/lib", "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10_hip", "-lc10", f"-L{PKG}", "-lmq",
           "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        if os.path.exists(out):
            os.remove(out)                                # it was built for another libmq.so
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stderr}")
    os.replace(out + ".tmp", out)
    return out


def build(verbose: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(lambda kv: _compile(*kv), SOURCES.items()))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    binding = _binding()
    if verbose:
        print(f"built {LIB} and {binding}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
