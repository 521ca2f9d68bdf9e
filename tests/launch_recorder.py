"""Host programs that call a launch interface of the library (csrc/*.h) with a HIP runtime that only records:
["limit", kernel, bytes] where a kernel's dynamic LDS limit is set, ["launch", kernel, dynamic LDS bytes, grid x, grid y,
threads] for a launch.  No GPU, and no device code."""
import json
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_prefill_ffn_amd", "csrc")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

RUNTIME = r"""
#include <cstdio>

extern "C" {
void** __hipRegisterFatBinary(const void*) { static void* m; return &m; }
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, dim3*, dim3*, int*) {}
void __hipUnregisterFatBinary(void**) {}
static struct { dim3 g, b; size_t lds; hipStream_t st; } cfg;
hipError_t __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, hipStream_t st) { cfg = {g, b, lds, st}; return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3* g, dim3* b, size_t* lds, hipStream_t* st)
{
    *g = cfg.g, *b = cfg.b, *lds = cfg.lds, *st = cfg.st;
    return hipSuccess;
}
hipError_t hipGetLastError(void) { return hipSuccess; }
static const char* sep = "";
hipError_t hipFuncSetAttribute(const void* f, hipFuncAttribute, int v)
{
    std::printf("%s[\"limit\", \"%p\", %d]", sep, f, v), sep = ", ";
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* f, dim3 g, dim3 b, void**, size_t lds, hipStream_t)
{
    std::printf("%s[\"launch\", \"%p\", %zu, %u, %u, %u]", sep, f, lds, g.x, g.y, b.x), sep = ", ";
    return hipSuccess;
}
}

"""


def record(at, header, source, main):
    """The events of `main`, a main() that includes `header` and calls into `source`."""
    if not shutil.which(HIPCC):
        pytest.skip("no hipcc")
    src, exe, objs = at / "main.hip", at / "main", []
    src.write_text(f'#include "{header}"' + RUNTIME + main)
    for s in (str(src), os.path.join(CSRC, source)):
        objs.append(str(at / (os.path.basename(s) + ".o")))
        r = subprocess.run([HIPCC, "--offload-host-only", "-std=c++17", "-O1", "-fPIC", "-I", CSRC, "-c", s, "-o", objs[-1]],
                           capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
    # what the program never calls (the device code, kernels of other sources) stays unresolved
    r = subprocess.run(["g++", *objs, "-Wl,--unresolved-symbols=ignore-all", "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    return json.loads(r.stdout)
