"""Compile libwq.so (HIP kernels + C ABI) in-tree for gfx950 with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libwq.so")
CALLS = os.path.join(HERE, "_calls.so")  # the compiled part of the Python binding
BUILD = os.path.join(HERE, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

COMMON = [
    "--offload-arch=gfx950", "-O3", "-fPIC", "-std=c++17",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]
# Quantization/packing/dequantization must be bit-exact: no contraction.
PER_FILE = {
    "wq_quant.hip": ["-ffp-contract=off"],
    "wq_gemv.hip": [],
    "wq_gemm.hip": [],
    # the probe's loop-carried MFMA accumulators stay in place only in the
    # VGPR form (the default AGPR form rotates them through copies every turn)
    "wq_probe.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
    "wq_noalloc.hip": [],
    "wq_rope.hip": [],
    "wq_kv_attn.hip": [],
    "wq_kv_chunk.hip": [],
    "wq_prompt_attn.hip": [],
    "wq_kv_tree.hip": [],
    # its codes too are whole numbers, one rounding an operation
    "wq_kv_append.hip": ["-ffp-contract=off"],
    "wq_verify.hip": [],
    "wq_api.cpp": [],
}


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *COMMON, *PER_FILE[os.path.basename(src)], "-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed for {src}")
    return obj


def build_calls(verbose: bool = False) -> str:
    """The compiled part of the Python binding, from torch's headers."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cmd = ["g++", "-O2", "-fPIC", "-std=c++17", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-isystem{d}" for d in (os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                                      sysconfig.get_paths()["include"])),
           os.path.join(CSRC, "wq_calls.cpp"), "-o", CALLS + ".tmp", "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu",
           "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("g++ failed for wq_calls.cpp")
    os.replace(CALLS + ".tmp", CALLS)
    return CALLS


def build(verbose: bool = False) -> str:
    """libwq.so.  hipcc is all that it takes: the C ABI is there without torch."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = [os.path.join(CSRC, f) for f in PER_FILE]
    with ThreadPoolExecutor(max_workers=min(4, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose=True))
    import importlib.util
    if importlib.util.find_spec("torch"):
        print(build_calls(verbose=True))
    else:
        print("torch is not installed: the Python binding is left out", file=sys.stderr)
