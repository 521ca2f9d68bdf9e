"""The struct layouts that a C compiler gives the 16-bit experts' and the adapters' part of include/moe_prefill.h equal
the binding's field by field, a C99 program can call them, and which kernels a call launches, by the launches that a
recording HIP runtime sees at the borders of each rule."""
import ctypes
import json
import os
import subprocess

import pytest

import moe_prefill_ffn_amd as mp
from launch_recorder import record

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIBDIR = os.path.join(ROOT, "moe_prefill_ffn_amd")
STRUCTS = ["moe_group_args_t", "moe_grouped_gemm_args_t", "moe_combine_args_t", "moe_lora_args_t"]


def test_c_layouts_and_calls(tmp_path):
    mp.lib()                                              # the library must be built
    lines = ["#include <moe_prefill.h>", "#include <stddef.h>", "#include <stdio.h>", "#include <string.h>", "int main(void) {", 'printf("{\\"v\\": 1");']
    for name in STRUCTS:
        lines.append(f'printf(", \\"{name}\\": [%zu", sizeof({name}));')
        lines += [f'printf(", %zu", offsetof({name}, {f}));' for f, _ in getattr(mp, name)._fields_]
        lines.append('printf("]");')
    lines += ["moe_group_args_t g; memset(&g, 0, sizeof g); g.struct_size = sizeof g; g.n_groups = 3;",
              "moe_grouped_gemm_args_t a; memset(&a, 0, sizeof a); a.struct_size = sizeof a; a.K = 8; a.N = a.n_groups = a.top_k = 1; a.dtype = MOE_BF16;",
              "moe_combine_args_t c; memset(&c, 0, sizeof c); c.struct_size = sizeof c; c.N = c.top_k = 1;",
              "moe_lora_args_t l; memset(&l, 0, sizeof l); l.struct_size = sizeof l; l.K = l.rank = 8; l.N = l.n_adapters = 1; l.dtype = MOE_F16;",
              "uint64_t gb = 1, lb = 1;",
              'printf(", \\"rc\\": [%d, %d, %d, %d, %d, %d]", moe_group_rows(&g, NULL), moe_grouped_gemm(&a, NULL), moe_combine_rows(&c, NULL),',
              "moe_lora_add(&l, NULL), moe_group_workspace_size(5000, 7, &gb), moe_lora_workspace_size(100, 64, 8, &lb));",
              'printf(", \\"bytes\\": [%llu, %llu]}\\n", (unsigned long long)gb, (unsigned long long)lb); return 0; }']
    src, exe = tmp_path / "client.c", tmp_path / "client"
    src.write_text("\n".join(lines))
    r = subprocess.run(["gcc", "-std=c99", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-L", LIBDIR,
                        "-l:libmoe_prefill.so", f"-Wl,-rpath,{LIBDIR}", "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    got = json.loads(r.stdout)
    for name in STRUCTS:
        cls = getattr(mp, name)
        assert got[name] == [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_], name
    # no bounds, no rows, no tokens, no rows, sizes
    assert got["rc"] == [mp.MOE_EINVAL] + [mp.MOE_OK] * 5
    assert got["bytes"] == [mp.moe_group_workspace_size(5000, 7), mp.moe_lora_workspace_size(100, 64, 8)]


@pytest.mark.parametrize("name,call", [("moe_group_args_t", "moe_group_rows"), ("moe_grouped_gemm_args_t", "moe_grouped_gemm"),
                                       ("moe_combine_args_t", "moe_combine_rows"), ("moe_lora_args_t", "moe_lora_add")])
def test_structs_of_another_header(name, call):
    cls = getattr(mp, name)

    class newer(ctypes.Structure):
        _fields_ = [("known", cls), ("later", ctypes.c_uint64)]

    for tail in (0, 1):
        n = newer()
        n.known.struct_size, n.later = ctypes.sizeof(n), tail
        rc = getattr(mp.lib(), call)(ctypes.cast(ctypes.byref(n), ctypes.POINTER(cls)), None)
        assert rc == mp.MOE_EINVAL
        assert ("struct" in mp.moe_prefill_last_error()) == (tail == 1)
    assert getattr(mp.lib(), call)(None, None) == mp.MOE_EINVAL


# ----------------------------------------------------------------- products ---

GEMM = r"""
int main()
{
    static uint8_t none[256];
    std::printf("[");
    const int sizes[][5] = {SIZES};                       // M, N, K, groups (0: dense), swiglu
    for (auto& s : sizes) {
        moe::Gemm16 g{};
        g.a = g.b = none, g.out = none;
        g.a_rows = g.M = s[0], g.N = s[1], g.K = s[2], g.row_div = 1, g.swiglu = s[4], g.out_stride = s[1];
        g.a_stride = g.b_stride = s[2] * 2, g.in_type = g.out_type = moe::kBF16;
        if (s[2] == 8) g.a_stride = 1 << 25;              // rows that span more than 32 bits of offset reach
        g.G = s[3] ? s[3] : 1, g.bounds = s[3] ? reinterpret_cast<const int32_t*>(none) : nullptr;
        if (launch_gemm16(g, 0) != hipSuccess) return 1;
    }
    std::printf("]\n");
    return 0;
}
"""
# LDS of a shape: its slots of (rows + columns of B) 128-byte rows
SHAPE = {"64": 8 * 128 * 128, "64x128": 6 * 192 * 128, "128 deep": 4 * 256 * 128, "128": 2 * 256 * 128, "128x256": 3 * 384 * 128, "256": 2 * 512 * 128}
RULE = [((1, 4096, 4096, 0, 0), "few 16"), ((16, 4096, 4096, 0, 0), "few 16"), ((17, 4096, 4096, 0, 0), "few 32"), ((32, 4096, 4096, 0, 0), "few 32"),
        ((33, 4096, 4096, 0, 0), "64"), ((64, 1024, 2048, 0, 0), "few 16"), ((256, 4096, 4096, 0, 0), "64"), ((512, 4096, 4096, 0, 0), "64x128"),
        ((1024, 4096, 4096, 0, 0), "128 deep"), ((2048, 4096, 4096, 0, 0), "128x256"), ((5000, 4096, 4096, 0, 0), "128"),
        ((8192, 4096, 4096, 0, 0), "256"), ((32, 1536, 4096, 0, 1), "few 16 swiglu"), ((33, 1536, 4096, 0, 1), "few 16 swiglu"),
        ((65, 1536, 4096, 0, 1), "64x128"), ((8, 768, 2048, 128, 1), "few 16 swiglu"), ((24, 768, 2048, 128, 1), "few 16 swiglu"),
        ((25, 768, 2048, 128, 1), "64x128"), ((8192, 768, 2048, 128, 1), "128x256"), ((16, 2048, 768, 128, 0), "few 32"), ((32, 2048, 768, 128, 0), "64x128"),
        ((65536, 4096, 1536, 256, 0), "128x256"), ((5000, 4096, 8, 0, 0), "few 32")]


@pytest.fixture(scope="module")
def gemm_events(tmp_path_factory):
    main = GEMM.replace("SIZES", ", ".join("{%d, %d, %d, %d, %d}" % s for s, _ in RULE))
    # one source a type: the fp16 one is not called and stays unresolved
    return record(tmp_path_factory.mktemp("launches"), "moe_gemm16.h", "moe_gemm16_bf16.hip", main)


def test_the_rule_of_the_shapes(gemm_events):
    launches = [e for e in gemm_events if e[0] == "launch"]
    assert len(launches) == len(RULE)
    for ((M, N, K, G, sw), shape), (_, _, lds, gx, gy, threads) in zip(RULE, launches):
        if shape.startswith("few"):
            cols = 32 if "32" in shape else 16
            rows = 32 if sw and not G and M > 32 else 16
            assert (threads, lds, gy) == (512, 0, -(-N // cols)), (M, N, K, shape)
            assert gx == (min(M, M // rows + G) if G else -(-M // rows))
        else:
            data = SHAPE[shape]
            assert threads == 256 and data < lds <= data + 8192, (M, N, K, shape, lds)
            assert gx % 8 == 0 and gx <= 256 * (160 * 1024 // lds)


def test_every_product_is_within_its_kernels_limit(gemm_events):
    limit = {}
    for kind, f, v, *_ in gemm_events:
        if kind == "limit":
            assert limit.setdefault(f, v) == v and v <= 160 << 10
        else:
            assert v <= limit.get(f, 0)


# ----------------------------------------------------- row table, adapters ---

GROUP = r"""
int main()
{
    static int none[64];
    std::printf("[");
    for (long long n : {0LL, 1LL, 4096LL, 4097LL, 65536LL, 300000LL, 1LL << 27}) {
        moe::GroupRows g{};
        g.eidx = g.bounds = g.rows = g.pos = g.ws = none;
        g.pairs = n, g.E = 1024;
        if (launch_group_rows(g, 0) != hipSuccess) return 1;
    }
    std::printf("]\n");
    return 0;
}
"""


def test_launches_of_the_row_table(tmp_path):
    events = record(tmp_path, "moe_rows.h", "moe_rows.hip", GROUP.replace("g.eidx = g.bounds", "g.eidx = none, g.bounds"))
    blocks = [e[3] for e in events if e[0] == "launch"]
    assert blocks == [1, 1, 1, 5, 5, 64, 64, 147, 147, 256, 256]
    for e in events:
        assert e[0] == "limit" and e[2] <= 160 << 10 or e[0] == "launch" and e[2] <= 70000 and e[5] == 1024
    for n, b in ((4097, 5), (65536, 64), (300000, 147), (1 << 27, 256)):
        assert mp.moe_group_workspace_size(n, 1024) == b * 4096


LORA = r"""
int main()
{
    static uint8_t none[256];
    std::printf("[");
    const int sizes[][5] = {SIZES};                       // M, K, N, r, fp32 base and out
    for (auto& s : sizes) {
        moe::LoraAdd l{};
        l.x = l.a = l.b = none, l.adapters = reinterpret_cast<const int32_t*>(none), l.base = l.out = none, l.ws = reinterpret_cast<float*>(none);
        l.M = s[0], l.K = s[1], l.N = s[2], l.r = s[3], l.n = 4, l.in_type = moe::kBF16;
        l.x_stride = 2 * l.K, l.base_stride = l.out_stride = l.N, l.base_type = l.out_type = s[4] ? moe::kF32 : moe::kBF16;
        if (launch_lora_add(l, 0) != hipSuccess) return 1;
    }
    std::printf("]\n");
    return 0;
}
"""
# the kernels' threads: one launch of 512, or 256 and 256 (few rows), 256 and 512 (many)
LORA_RULE = [((1, 4096, 4096, 16, 0), [512]), ((1, 4096, 4096, 40, 0), [256, 256]), ((16, 4096, 4096, 16, 0), [512]), ((64, 4096, 4096, 16, 0), [256, 256]),
             ((64, 2048, 2048, 16, 0), [512]), ((1024, 4096, 4096, 16, 0), [256, 256]), ((1025, 4096, 4096, 16, 0), [256, 512]), ((1025, 4096, 4095, 16, 0), [256, 256]),
             ((8192, 4096, 4096, 64, 0), [256, 512]), ((8192, 4096, 4096, 256, 1), [256, 512]), ((8192, 64, 64, 8, 1), [256, 512])]


def test_launches_of_the_adapters(tmp_path):
    main = LORA.replace("SIZES", ", ".join("{%d, %d, %d, %d, %d}" % s for s, _ in LORA_RULE))
    events = record(tmp_path, "moe_lora.h", "moe_lora.hip", main)
    launches = [e for e in events if e[0] == "launch"]
    assert [e[5] for e in launches] == [t for _, ts in LORA_RULE for t in ts]
    limit = {e[1]: e[2] for e in events if e[0] == "limit"}
    for e in launches:
        assert e[2] <= limit.get(e[1], 0) <= 160 << 10
        assert e[3] * e[5] < 1 << 32 and e[4] < 65536
