"""Build libttt.so (the HIP kernels and the C ABI) for gfx950 with hipcc and, for Python, _seq_native.so (seq.py's
marshalling) with g++ against PyTorch, in-tree. libttt.so needs hipcc alone.

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


def native_command(out: str):
    """g++ on seq_native.cpp: host code only, against PyTorch's headers and libraries (which the process that
    loads the module has loaded already). None where there is no PyTorch."""
    spec = importlib.util.find_spec("torch")  # (found, not imported)
    if spec is None or spec.origin is None:
        return None
    torch = os.path.dirname(spec.origin)
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-I", os.path.join(ROOT, "include"),
            "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"], "-Wall", "-Wextra",
            os.path.join(CSRC, "seq_native.cpp"), "-o", out, "-L", os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10", "-lc10_hip"]


def flags_for(src: str) -> list:
    return FLAGS + SOURCE_FLAGS.get(src, [])


def _start(cmd):
    """The command's process, or what kept it from starting."""
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    except OSError as e:
        return str(e)


def _end(p):
    """Waits for a started command: (it succeeded, what it said)."""
    if isinstance(p, str):
        return False, p
    out = p.communicate()[0]
    # hipcc's host pass warns that it does not know the packed-fp32 feature; drop that noise.
    return p.returncode == 0, "\n".join(ln for ln in out.splitlines() if "packed-fp32-ops" not in ln)


def _put(tmp, path):
    """tmp in path's place, or, without a tmp, neither of them."""
    if tmp is not None:
        os.replace(tmp, path)
    else:
        for f in (path, path + ".tmp"):
            if os.path.exists(f):
                os.remove(f)


def build(verbose: bool = False) -> str:
    """Compile every source and link libttt.so and, where there is PyTorch, _seq_native.so; returns libttt.so's path.
    Raises on failure: of a HIP source with what was built before left as it was, of the binding with libttt.so in
    place and no binding."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    objs = [os.path.join(BUILD_DIR, src.replace(".hip", ".o")) for src in SOURCES]
    procs = [_start([HIPCC, *flags_for(src), "-c", os.path.join(CSRC, src), "-o", obj]) for src, obj in zip(SOURCES, objs)]
    native, tmp = NATIVE + ".tmp", LIB + ".tmp"
    command = native_command(native)
    binding = _start(command) if command else None
    said = [(src, *_end(p)) for src, p in zip(SOURCES, procs)]  # (all of them: none is left running)
    bound, bound_said = _end(binding) if command else (False, "")
    for src, ok, out in said:
        if not ok:
            if os.path.exists(native):
                os.remove(native)
            raise RuntimeError(f"the compiler failed on {src}:\n{out}")
        if verbose and out.strip():
            print(out)
    ok, out = _end(_start([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]))
    if not ok:
        if os.path.exists(native):
            os.remove(native)
        raise RuntimeError(f"link failed:\n{out}")
    _put(tmp, LIB)
    _put(native if bound else None, NATIVE)
    if not command:
        print("no PyTorch: _seq_native.so (the block operators' Python binding) is left out", file=sys.stderr)
    elif not bound:
        raise RuntimeError(f"the compiler failed on seq_native.cpp:\n{bound_said}")
    elif verbose and bound_said.strip():
        print(bound_said)
    return LIB


if __name__ == "__main__":
    path = build(verbose="-v" in sys.argv)
    print(path)
