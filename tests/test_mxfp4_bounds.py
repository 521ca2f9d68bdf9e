"""Group bounds beyond [0, M]: the product is the one of the clamped bounds, in the few-row and the tiled kernels."""
import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref
from test_mxfp4 import check_product, gen, random_mx

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K", [(40, 64, 64), (100, 33, 288), (180, 40, 512), (700, 64, 96), (3000, 200, 512)])
def test_ascending_bounds_are_clamped(M, N, K, swiglu):
    g = gen(M + N)
    cases = [[-7, 2, M // 2, M], [-40, -3, 5, M + 9], [-(1 << 31), 10, 10, (1 << 31) - 1], [-70, 30, 35, M - 5], [-33, -1, M // 3, M + 1000],
             [5, M // 2, M, M + 64], [-64, -32, 0, 32], [M - 1, M + 1, M + 2, M + 3], [-5, -4, -3, -2], [M, M + 1, M + 40, M + 90]]
    a, b = random_mx(g, M, K, hi=120), random_mx(g, 3, 2 * N if swiglu else N, K, hi=120)
    ad, bd = [t.cuda() for t in a], [t.cuda() for t in b]
    for bounds in cases:
        out = torch.full((M, N), 77.0, device="cuda")
        mp.moe_mxfp4_gemm(*ad, *bd, out, bounds=torch.tensor(bounds).int().cuda(), swiglu=swiglu)
        torch.cuda.synchronize()
        clamped = torch.tensor(bounds).clamp(0, M)
        want, err = ref.mx_product(ref.mx_values(*a), ref.mx_values(*b), clamped, swiglu=swiglu)
        lo, hi = int(clamped[0]), int(clamped[-1])
        assert (out[:lo] == 77).all() and (out[hi:] == 77).all(), bounds
        if hi > lo:
            check_product(out[lo:hi], torch.float32, want[lo:hi], err[lo:hi])
