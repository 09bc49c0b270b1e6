"""Build libq4moe.so in-tree for gfx950 with hipcc.

``python -m quantized_moe_expert_q4_amd.build`` (or ``build()``) compiles the
HIP kernels and the C ABI into ``quantized_moe_expert_q4_amd/libq4moe.so``.
"""
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libq4moe.so")

SOURCES = ["q4moe_resident.hip", "q4moe_batch.hip", "q4moe_chunked.hip", "q4moe_stream.hip", "q4moe_sigmoid.hip", "q4moe_noalloc.hip",
           "q4moe_linear.hip", "q4moe_linear32.hip", "q4moe_linear64.hip", "q4moe_linear128.hip",
           "q4moe_linear_back.hip", "q4moe_adapter.hip", "q4moe_adapter_grad.hip",
           "q4moe_route.hip", "q4moe_combine.hip", "q4moe_abi.cpp", "q4moe_layer_abi.cpp"]

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-ffp-contract=off",
    # packed-FP32 instructions are kept out of every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libq4moe.so)")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                    if "is not a recognized feature for this target" not in l)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + out)
    if out.strip() and verbose:
        print(out)


def build(verbose: bool = False) -> str:
    """Compile every source to an object (in parallel), then link the library."""
    cc = hipcc()
    with tempfile.TemporaryDirectory(prefix="q4moe_build_") as tmpdir:
        objs = [os.path.join(tmpdir, os.path.splitext(s)[0] + ".o") for s in SOURCES]
        cmds = [[cc, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, s), "-o", o]
                for s, o in zip(SOURCES, objs)]
        with ThreadPoolExecutor(max_workers=len(cmds)) as ex:
            for f in [ex.submit(_run, c, verbose) for c in cmds]:
                f.result()
        tmp = LIB + ".tmp"
        _run([cc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
