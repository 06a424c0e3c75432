"""Build libmnb.so (HIP, gfx950) in-tree with hipcc.

    python blockwise_bit_quantized_amd/build.py

(run by path: importing the package loads the library this script builds)
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libmnb.so")
# measurement helper for the benchmark (a streaming-read ceiling kernel), not the ABI
CEILING_LIB = os.path.join(PKG, "libmnb_ceiling.so")
CEILING_SOURCE = "ceiling.hip"
# host side of the torch binding of include/mnb_ops.h (built where torch is installed)
BINDING_LIB = os.path.join(PKG, "_mnb_ops" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
BINDING_SOURCE = "binding.cpp"
OBJ = os.path.join(PKG, "_build")
SOURCES = ["api.hip", "gemv.hip", "gemv_mfma.hip", "gemv_acc4.hip", "tproj.hip", "gemm.hip", "pack.hip",
           "api_ops.hip", "mx_quant.hip", "mx_gemv.hip", "mx_gemm.hip", "rmsnorm.hip", "logprobs.hip",
           "api_decode.hip", "kv_append.hip", "kv_attention.hip", "sample.hip"]
ARCH = os.environ.get("MNB_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    "--offload-arch=" + ARCH, "-O3", "-std=c++17", "-fPIC", "-Wall",
    # code object v5 loads under both the system ROCm runtime and the one torch bundles
    "-mcode-object-version=5",
    # packed FP32 ops are disabled for every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
]


def _hipcc() -> str:
    for c in (os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "bin", "hipcc"), "hipcc"):
        if os.path.sep not in c or os.path.exists(c):
            return c
    return "hipcc"


def build(verbose: bool = False, jobs: int = 8) -> str:
    os.makedirs(OBJ, exist_ok=True)
    hipcc = _hipcc()

    def compile_one(src):
        obj = os.path.join(OBJ, src.replace(".hip", ".o"))
        cmd = [hipcc, *HIPCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        err = "\n".join(l for l in r.stderr.splitlines() if "packed-fp32-ops" not in l)
        if r.returncode != 0:
            raise RuntimeError("hipcc failed for %s:\n%s" % (src, err))
        if err.strip() and verbose:
            print(err, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=min(jobs, len(SOURCES) + 1)) as ex:
        binding = ex.submit(_build_binding, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc, "--offload-arch=" + ARCH, "-mcode-object-version=5", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr)
    _check_undefined(tmp)
    os.replace(tmp, LIB)
    _build_ceiling(hipcc, verbose)
    return LIB


def _build_binding(verbose: bool) -> None:
    """The torch module.  Where its tools are not there the library stands alone: MatMulNBits and the C ABI
    need nothing else, and the torch calls of the operators raise an ImportError."""
    spec = importlib.util.find_spec("torch")
    torch = os.path.join(list(spec.submodule_search_locations)[0]) if spec else ""
    inc, lib = os.path.join(torch, "include"), os.path.join(torch, "lib")
    python = sysconfig.get_paths()["include"]
    missing = ["torch"] if spec is None else [
        what for what, there in (("g++", shutil.which("g++")),
                                 ("torch's headers", os.path.exists(os.path.join(inc, "ATen", "ATen.h"))),
                                 ("Python's headers", os.path.exists(os.path.join(python, "Python.h")))) if not there]
    if missing:
        if os.path.exists(BINDING_LIB):          # of an earlier build: not of this library
            os.remove(BINDING_LIB)
        print("_mnb_ops is not built: no %s" % " and no ".join(missing), file=sys.stderr, flush=True)
        return
    tmp = BINDING_LIB + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-DUSE_ROCM", "-D__HIP_PLATFORM_AMD__=1",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", python, "-I" + os.path.join(ROOT, "include"),
           os.path.join(CSRC, BINDING_SOURCE), "-o", tmp, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s" % (BINDING_SOURCE, r.stderr))
    os.replace(tmp, BINDING_LIB)


def _build_ceiling(hipcc: str, verbose: bool) -> None:
    tmp = CEILING_LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc, *HIPCC_FLAGS, "-shared", os.path.join(CSRC, CEILING_SOURCE), "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (CEILING_SOURCE, r.stderr))
    os.replace(tmp, CEILING_LIB)


def _check_undefined(path: str) -> None:
    """A kernel whose host-side launch stub was not emitted links fine but cannot be
    loaded; refuse such a library here instead of at import time."""
    r = subprocess.run(["nm", "-D", "--undefined-only", path], capture_output=True, text=True)
    if r.returncode != 0:
        return                                   # nm unavailable: the loader still checks
    bad = [l.split()[-1] for l in r.stdout.splitlines() if "_ZN3mnb" in l]
    if bad:
        os.remove(path)
        raise RuntimeError("libmnb links against undefined symbols of its own: " + ", ".join(bad[:4]))


if __name__ == "__main__":
    print(build(verbose=True))
    sys.exit(0)
