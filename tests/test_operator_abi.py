"""The struct layouts that a C compiler gives the few-token layer's and the MXFP4 operators' part of
include/moe_prefill.h equal the binding's field by field, a C99 program can call them, and a struct of
a newer header is taken only where its unknown tail is zero."""
import ctypes
import json
import os
import subprocess

import pytest

import moe_prefill_ffn_amd as mp

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "moe_prefill_ffn_amd")
STRUCTS = ["moe_decode_io_t", "moe_mxfp4_matrix_t", "moe_mxfp4_gemm_args_t"]


def test_c_layouts_and_calls(tmp_path):
    mp.lib()                                              # the library must be built
    lines = ["#include <moe_prefill.h>", "#include <stddef.h>", "#include <stdio.h>", "#include <string.h>", "int main(void) {",
             'printf("{\\"consts\\": [%d, %d, %d, %d]", MOE_F32, MOE_BF16, MOE_F16, MOE_DECODE_MAX_PAIRS);']
    for name in STRUCTS:
        lines.append(f'printf(", \\"{name}\\": [%zu", sizeof({name}));')
        lines += [f'printf(", %zu", offsetof({name}, {f}));' for f, _ in getattr(mp, name)._fields_]
        lines.append('printf("]");')
    lines += ["moe_mxfp4_matrix_t m; memset(&m, 0, sizeof m); m.struct_size = sizeof m; m.K = 32;",
              "moe_mxfp4_gemm_args_t a; memset(&a, 0, sizeof a); a.struct_size = sizeof a; a.K = 32; a.N = a.n_groups = a.top_k = 1;",
              "moe_decode_io_t io; memset(&io, 0, sizeof io); io.struct_size = sizeof io;",
              "moe_prefill_params_t p; memset(&p, 0, sizeof p); p.struct_size = sizeof p; uint64_t bytes = 0;",
              "p.d_model = p.d_ff = 64; p.n_experts = 4; p.top_k = 2; p.max_tokens = 1;",
              'printf(", \\"rc\\": [%d, %d, %d, %d, %d]", moe_mxfp4_quantize(&m, NULL), moe_mxfp4_dequantize(&m, NULL),',
              "moe_mxfp4_gemm(&a, NULL), moe_decode_run_layer(NULL, &io, NULL), moe_decode_workspace_size(&p, &bytes));",
              'printf(", \\"bytes\\": %llu}\\n", (unsigned long long)bytes); return 0; }']
    src, exe = tmp_path / "client.c", tmp_path / "client"
    src.write_text("\n".join(lines))
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-L", LIBDIR,
                        "-l:libmoe_prefill.so", f"-Wl,-rpath,{LIBDIR}", "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    got = json.loads(r.stdout)
    assert got["consts"] == [mp.MOE_F32, mp.MOE_BF16, mp.MOE_F16, mp.MOE_DECODE_MAX_PAIRS]
    for name in STRUCTS:
        cls = getattr(mp, name)
        assert got[name] == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_], name
    # no rows, no rows, no rows, no handle, a size
    assert got["rc"] == [mp.MOE_OK, mp.MOE_OK, mp.MOE_OK, mp.MOE_EINVAL, mp.MOE_OK]
    assert got["bytes"] == mp.moe_decode_workspace_size(64, 64, 4, 2, 1)


@pytest.mark.parametrize("tail,code", [(0, mp.MOE_OK), (1, mp.MOE_EINVAL)])
def test_structs_of_a_newer_header(tail, code):
    class newer(ctypes.Structure):
        _fields_ = [("known", mp.moe_mxfp4_matrix_t), ("later", ctypes.c_uint64)]

    n = newer()
    n.known.struct_size = ctypes.sizeof(n)
    n.known.K, n.later = 32, tail
    p = ctypes.cast(ctypes.byref(n), ctypes.POINTER(mp.moe_mxfp4_matrix_t))
    assert mp.lib().moe_mxfp4_quantize(p.contents, None) == code


@pytest.mark.parametrize("call", ["moe_mxfp4_quantize", "moe_mxfp4_dequantize"])
@pytest.mark.parametrize("K", [32, 96, 1 << 20])
def test_the_largest_matrix_of_one_launch(call, K):
    """The last size whose workgroups of 64 blocks, 256 threads each, stay below 2^32 threads is taken (the call
    then misses its pointers), the next one is not."""
    def message(M):
        m = mp.moe_mxfp4_matrix_t(struct_size=ctypes.sizeof(mp.moe_mxfp4_matrix_t), K=K, M=M, stride=K)
        assert getattr(mp.lib(), call)(m, None) == mp.MOE_EINVAL
        return mp.moe_prefill_last_error()

    nb = K // 32
    most = max(M for M in range((1 << 30) // nb - 100, (1 << 30) // nb + 1) if -(-M * nb // 64) * 256 < 1 << 32)
    assert "required" in message(most)
    assert "2^30" in message(most + 1) and "2^30" in message(most + 63 // nb + 1)
