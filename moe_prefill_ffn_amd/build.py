"""Build libmoe_prefill.so (HIP for gfx950 + the host runtime) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoe_prefill.so")
MICRO_LIB = os.path.join(HERE, "libmoe_micro.so")   # measurement kernels (roofline denominators)
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

SOURCES = ["moe_mx.hip", "moe_gemm16_bf16.hip", "moe_gemm16_f16.hip", "moe_kernels.hip", "moe_decode.hip", "moe_lora.hip", "moe_rows.hip",
           "moe_runtime.cpp", "moe_pack.cpp", "moe_pool_plan.cpp"]

# -ffp-contract=off: no fused multiply-adds beyond the ones written out.
# No fast-math: IEEE division (correctly rounded), fp32 denormals kept.
# -packed-fp32-ops: keep the compiler off the packed fp32 VALU instructions.
ARCH = "--offload-arch=gfx950"
FLAGS = [
    ARCH, "-O3", "-fPIC", "-std=c++17",
    "-ffp-contract=off", "-fno-fast-math",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
    "-Wno-inline-asm",   # M0 is clobbered on purpose by the direct-to-LDS loads (no compiler use of M0 there)
]


def _run(cmd, what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"hipcc failed building {what}")


def _hipcc(sources, out: str, verbose: bool) -> None:
    """Each source to an object, at once, then the library from them."""
    tmp = out + ".tmp"
    with tempfile.TemporaryDirectory() as objs:
        def compile_one(s):
            o = os.path.join(objs, s + ".o")
            _run([HIPCC] + FLAGS + ["-c", os.path.join(CSRC, s), "-o", o], s, verbose)
            return o

        with ThreadPoolExecutor(max_workers=min(len(sources), os.cpu_count() or 1)) as pool:
            made = list(pool.map(compile_one, sources))
        _run([HIPCC, ARCH, "-shared", "-fPIC"] + made + ["-o", tmp], os.path.basename(out), verbose)
    os.replace(tmp, out)


def build(verbose: bool = False) -> str:
    _hipcc(SOURCES, LIB, verbose)
    _hipcc(["moe_micro.hip"], MICRO_LIB, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
