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
        std::printf("%s[\"case\"]", sep), sep = ", ";
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
LARGEST = [(1 << 27, 2, 8, 0, 0, 1 << 25), (1 << 27, 256, 8, 0, 0, 1 << 25), (1 << 27, 100, 8, 65535, 1, 1 << 25), (1 << 27, 256, 8, 0, 0, 0),
           (1 << 27, 32, 8, 65535, 0, 0), (1, 1 << 20, 8, 0, 1, 0), (24, 1 << 20, 64, 300, 1, 0), (4, 1 << 20, 8, 0, 0, 0), (1000, 1 << 20, 64, 0, 0, 1 << 25)]


def launches_of(at, sizes):
    """The launches of each of the sizes, in their order."""
    out = []
    for e in record(at, "moe_gemm16.h", "moe_gemm16_bf16.hip", LAUNCHES.replace("SIZES", ", ".join("{%d, %d, %d, %d, %d, %d}" % s for s in sizes))):
        if e[0] == "case":
            out.append([])
        elif e[0] == "launch":
            out[-1].append(e)
    assert len(out) == len(sizes)
    return out


def test_launches_hold_the_largest_calls(tmp_path):
    """Fewer than 2^32 threads along x and 65536 workgroups along y in every launch; few-row launches cover all tiles."""
    for (M, N, K, G, swiglu, b_stride), launches in zip(LARGEST, launches_of(tmp_path, LARGEST)):
        assert launches and all(gx * threads < 1 << 32 and gy < 65536 for _, _, _, gx, gy, threads in launches), (M, N, G)
        if launches[0][2] == 0:                           # no dynamic LDS: the few-row kernel
            tiles = [min(M, M // rows + G if G else -(-M // rows)) * -(-N // cols) for rows in (16, 32) for cols in (16, 32)]
            assert sum(gx * gy for _, _, _, gx, gy, _ in launches) in tiles, (M, N, G)


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


TABLES = r"""
int main()
{
    static uint8_t none[256];
    std::printf("[");
    const long long sizes[][6] = {SIZES};                 // M, N, K, rows of A, by a table, top_k
    for (auto& s : sizes) {
        moe::Gemm16 g{};
        g.a = g.b = none, g.out = none;
        g.M = s[0], g.N = (int)s[1], g.K = (int)s[2], g.a_rows = s[3], g.rows = s[4] ? reinterpret_cast<const int32_t*>(none) : nullptr, g.row_div = (int)s[5];
        g.a_stride = g.b_stride = s[2] * 2, g.out_stride = s[1], g.in_type = g.out_type = moe::kBF16, g.G = 1;
        if (launch_gemm16(g, 0) != hipSuccess) return 1;
    }
    std::printf("]\n");
    return 0;
}
"""


def test_many_rows_through_a_table_over_more_than_4_gib_are_tiled(tmp_path):
    """Up to 64 GiB; without a table a tile's own rows count, however many A has."""
    cases = [((8192, 4096, 4096, 524287, 1, 1), True), ((8192, 4096, 4096, 524289, 1, 1), True), ((8192, 4096, 4096, (1 << 23) - 1, 1, 8), True),
             ((8192, 4096, 4096, (1 << 23) + 1, 1, 8), False), ((1 << 21, 4096, 4096, 1 << 20, 0, 2), True)]
    events = record(tmp_path, "moe_gemm16.h", "moe_gemm16_bf16.hip", TABLES.replace("SIZES", ", ".join("{%d, %d, %d, %d, %d, %d}" % c for c, _ in cases)))
    launches = [e for e in events if e[0] == "launch"]
    assert [e[2] > 0 for e in launches] == [tiled for _, tiled in cases]
    # the kernel with whole addresses from 4 GiB on
    assert launches[0][1] == launches[4][1] != launches[1][1] == launches[2][1]


@gpu
@pytest.mark.parametrize("K", [256, 4096, 72])
@pytest.mark.parametrize("M,N,G,k,swiglu", [(3000, 300, 5, 1, False), (700, 200, 3, 4, True), (2500, 2100, 1, 2, False)])
def test_tiles_through_a_table_over_more_than_4_gib(M, N, G, k, swiglu, K):
    g = gen(M + K)
    A = (1 << 32) // (2 * K) + 1000
    a = torch.zeros(A, K, dtype=torch.bfloat16, device="cuda")
    ar = torch.tensor(sorted({0, 1, A // 3, A // 2 - 1, A - 1001, A - 1000, A - 999, A - 2, A - 1}))
    a[ar.cuda()] = normal(g, torch.bfloat16, len(ar), K).cuda()
    b = normal(g, torch.bfloat16, G, 2 * N if swiglu else N, K) / math.sqrt(K)
    near = torch.randint(0, len(ar), (M,), generator=g)
    rows = ar[near] * k + torch.randint(0, k, (M,), generator=g)
    bounds = torch.tensor([M * i // G for i in range(G + 1)]).int()
    out = mp.moe_grouped_gemm(a, b.cuda(), bounds=bounds.cuda(), rows=rows.int().cuda(), top_k=k, swiglu=swiglu, dtype=torch.float32)
    want, err = ref.mx_product(a[ar.cuda()].double(), b.double().cuda(), bounds, near, 1, swiglu)
    check_product(out, torch.float32, want.cpu(), err.cpu())


@gpu
@pytest.mark.parametrize("K,k", [(4096, 2), (128, 3)])
def test_copies_of_each_row_of_more_than_4_gib(K, k):
    """Without a table, top_k rows of the product a row of A: the last rows of A stand past 32 bits of offset."""
    g = torch.Generator(device="cuda").manual_seed(K)
    A, N = (1 << 32) // (2 * K) + 100, 8
    a = torch.zeros(A, K, dtype=torch.bfloat16, device="cuda")
    a[-300:] = torch.randn(300, K, generator=g, device="cuda")
    b = (torch.randn(N, K, generator=g, device="cuda") / math.sqrt(K)).bfloat16()
    out = mp.moe_grouped_gemm(a, b, top_k=k)
    want, err = ref.mx_product(a[-300:].double(), b.double()[None], None, None, k)
    check_product(out[-300 * k:], torch.bfloat16, want.cpu(), err.cpu())
    assert (out[:-300 * k] == 0).all()
