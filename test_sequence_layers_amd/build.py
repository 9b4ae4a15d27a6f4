"""Build libttt.so (the HIP kernels and the C ABI) for gfx950 with hipcc and _seq_native.so (seq.py's marshalling)
with g++, in-tree.

    python -m test_sequence_layers_amd.build
"""
from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libttt.so")
SOURCES = ["abi.hip", "fullbatch.hip", "chunked.hip", "mlp.hip", "dwconv.hip", "grid.hip", "epilogue.hip",
           "abi_seq.hip", "layernorm.hip", "conv1d.hip", "scan.hip"]
NATIVE = os.path.join(HERE, "_seq_native.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# Packed fp32 ops are disabled for all device code: hipcc would otherwise form v_pk_* fp32
# instructions from ordinary float code.
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
    "-Wno-unused-command-line-argument",
]
# Per-source additions. MFMA accumulators in ordinary VGPRs: otherwise the compiler parks them in
# AGPRs and moves them back and forth (v_accvgpr_read/write) around every conversion of a result.
# Measured: causal TTT-Linear 91 -> 86 us; the TTT-MLP kernel (no AGPR moves either way) is left
# as it was. The chunk-step kernels (chunked scans, TTT-MLP) are chains of dependent short
# operations; the scheduler's ILP-maximising strategy orders them slightly better (bidirectional
# 46.1 -> 45.1 us, TTT-MLP 958 -> 947-954 us; the full-batch kernels are unchanged by it). For the
# split TTT-MLP schedule: 0.815-0.819 ms, against 0.826 (default), 0.828 (max-memory-clause), 0.840
# (iterative-ilp) and 0.858 ms (iterative-minreg).
SCHED_ILP = ["-mllvm", "-amdgpu-sched-strategy=max-ilp"]
SOURCE_FLAGS = {
    "fullbatch.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
    "chunked.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1", *SCHED_ILP],
    "mlp.hip": SCHED_ILP,
    "scan.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"],
}


def native_command(out: str) -> list:
    """g++ on seq_native.cpp: host code only, against PyTorch's headers and libraries (which the process that
    loads the module has loaded already)."""
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)  # (found, not imported)
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-I", os.path.join(ROOT, "include"),
            "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"], "-Wall", "-Wextra",
            os.path.join(CSRC, "seq_native.cpp"), "-o", out, "-L", os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10", "-lc10_hip"]


def flags_for(src: str) -> list:
    return FLAGS + SOURCE_FLAGS.get(src, [])


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature; drop that noise.
    lines = [ln for ln in p.stdout.splitlines() if "packed-fp32-ops" not in ln]
    return p.returncode, "\n".join(lines)


def build(verbose: bool = False) -> str:
    """Compile every source and link libttt.so and _seq_native.so; returns libttt.so's path. Raises on failure."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        cmd = [HIPCC, *flags_for(src), "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    native = NATIVE + ".tmp"
    procs.append(("seq_native.cpp", None, subprocess.Popen(native_command(native), stdout=subprocess.PIPE,
                                                           stderr=subprocess.STDOUT, text=True)))
    objs = []
    for src, obj, p in procs:
        out, _ = p.communicate()
        out = "\n".join(ln for ln in out.splitlines() if "packed-fp32-ops" not in ln)
        if p.returncode != 0:
            raise RuntimeError(f"the compiler failed on {src}:\n{out}")
        if verbose and out.strip():
            print(out)
        if obj is not None:
            objs.append(obj)
    tmp = LIB + ".tmp"
    rc, out = _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs])
    if rc != 0:
        raise RuntimeError(f"link failed:\n{out}")
    os.replace(tmp, LIB)
    os.replace(native, NATIVE)
    return LIB


if __name__ == "__main__":
    path = build(verbose="-v" in sys.argv)
    print(path)
