"""16-bit products at the ends of what a call may ask for: what one launch holds, by a recording HIP runtime, and values."""
import math

import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref
from launch_recorder import record
from test_experts16 import normal
from test_mxfp4 import check_product, gen

gpu = pytest.mark.gpu

LAUNCHES = r"""
int main()
{
    static uint8_t none[256];
    std::printf("[");
    const long long sizes[][6] = {SIZES};                 // M, N, K, groups (0: dense), swiglu, bytes from a row of B to the next
    for (auto& s : sizes) {
        moe::Gemm16 g{};
        g.a = g.b = none, g.out = none;
        g.a_rows = g.M = s[0], g.N = (int)s[1], g.K = (int)s[2], g.row_div = 1, g.swiglu = (int)s[4], g.out_stride = s[1];
        g.a_stride = s[2] * 2, g.b_stride = s[5] ? s[5] : s[2] * 2, g.in_type = g.out_type = moe::kBF16;
        g.G = s[3] ? (int)s[3] : 1, g.bounds = s[3] ? reinterpret_cast<const int32_t*>(none) : nullptr;
        if (launch_gemm16(g, 0) != hipSuccess) return 1;
    }
    std::printf("]\n");
    return 0;
}
"""


@pytest.mark.parametrize("M,N,K,G,swiglu,b_stride", [
    (1 << 27, 2, 8, 0, 0, 1 << 25), (1 << 27, 256, 8, 0, 0, 1 << 25), (1 << 27, 100, 8, 65535, 1, 1 << 25), (1 << 27, 256, 8, 0, 0, 0), (1 << 27, 32, 8, 65535, 0, 0),
    (1, 1 << 20, 8, 0, 1, 0), (24, 1 << 20, 64, 300, 1, 0), (4, 1 << 20, 8, 0, 0, 0), (1000, 1 << 20, 64, 0, 0, 1 << 25)])
def test_launches_hold_the_largest_calls(tmp_path, M, N, K, G, swiglu, b_stride):
    """Fewer than 2^32 threads along x and 65536 workgroups along y in every launch; few-row launches cover all tiles."""
    events = record(tmp_path, "moe_gemm16.h", "moe_gemm16_bf16.hip", LAUNCHES.replace("SIZES", "{%d, %d, %d, %d, %d, %d}" % (M, N, K, G, swiglu, b_stride)))
    launches = [e for e in events if e[0] == "launch"]
    assert launches and all(gx * threads < 1 << 32 and gy < 65536 for _, _, _, gx, gy, threads in launches)
    if launches[0][2] == 0:                               # no dynamic LDS: the few-row kernel
        tiles = {(rows, cols): min(M, M // rows + G if G else -(-M // rows)) * -(-N // cols) for rows in (16, 32) for cols in (16, 32)}
        assert sum(gx * gy for _, _, _, gx, gy, _ in launches) in tiles.values()


@gpu
@pytest.mark.parametrize("M", [1, 3])
def test_the_most_columns_with_swiglu(M):
    """2^20 columns, 16 a workgroup."""
    g = gen(M)
    N, K = 1 << 20, 8
    a, b = normal(g, torch.bfloat16, M, K), normal(g, torch.bfloat16, 1, 2 * N, K) / math.sqrt(K)
    out = mp.moe_grouped_gemm(a.cuda(), b[0].cuda(), swiglu=True)
    want, err = ref.mx_product(a.double(), b.double(), swiglu=True)
    check_product(out, torch.bfloat16, want, err)


@gpu
def test_the_most_rows_by_the_few_row_kernel():
    """2^27 rows, against B whose rows stand more than 2^24 bytes apart."""
    M, N, K, step = 1 << 27, 2, 8, 1 << 24
    g = torch.Generator(device="cuda").manual_seed(1)
    a = torch.randn(M, K, generator=g, device="cuda", dtype=torch.bfloat16)
    b = torch.zeros(step + K, dtype=torch.bfloat16, device="cuda").as_strided((N, K), (step, 1))
    b.copy_(torch.randn(N, K, generator=g, device="cuda"))
    out = mp.moe_grouped_gemm(a, b)
    for i in range(0, M, 1 << 24):
        want, err = ref.mx_product(a[i:i + (1 << 24)].double(), b.double()[None])
        assert ((out[i:i + (1 << 24)].double() - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all()
