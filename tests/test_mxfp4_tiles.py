"""The widest tiles of the product, at the lengths of K that choose them, and next to their border."""
import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref
from test_mxfp4 import check_product, gen, groups_of, random_mx

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("K", [2784, 2816, 2880, 4096, 4608])   # below the border; scale rows 4-byte aligned, not, 16-byte
@pytest.mark.parametrize("M,N,swiglu,dtype", [(5000, 6100, False, torch.float32), (5001, 3050, True, torch.bfloat16),
                                              (4990, 6099, False, torch.float16)])
def test_dense(M, N, K, swiglu, dtype):
    g = gen(M + K)
    a = [t.cuda() for t in random_mx(g, M, K, hi=116)]
    b = [t.cuda() for t in random_mx(g, 2 * N if swiglu else N, K, hi=116)]
    out = torch.full((M + 2, N), 77.0, dtype=dtype, device="cuda")
    mp.moe_mxfp4_gemm(*a, *b, out[:M], swiglu=swiglu)
    want, err = ref.mx_product(ref.mx_values(*a).cuda(), ref.mx_values(*b)[None].cuda(), swiglu=swiglu)
    check_product(out[:M], dtype, want.cpu(), err.cpu())
    assert (out[M:] == 77).all()


@gpu
@pytest.mark.parametrize("kind", ["random", "part"])
@pytest.mark.parametrize("M,N,K,G,k,swiglu", [(6000, 5000, 2880, 8, 2, False), (5600, 4100, 4096, 12, 1, False), (5000, 2600, 2816, 9, 2, True)])
def test_grouped(kind, M, N, K, G, k, swiglu):
    g = gen(M + K)
    a, b = random_mx(g, M // k, K, hi=116), random_mx(g, G, 2 * N if swiglu else N, K, hi=116)
    bounds, rows = groups_of(kind, G, M, g), torch.randperm(M, generator=g).int()
    out = torch.full((M, N), 77.0, device="cuda")
    mp.moe_mxfp4_gemm(*[t.cuda() for t in a], *[t.cuda() for t in b], out, bounds=bounds.cuda(), rows=rows.cuda(), top_k=k, swiglu=swiglu)
    want, err = ref.mx_product(ref.mx_values(*a).cuda(), ref.mx_values(*b).cuda(), bounds, rows, k, swiglu)
    lo, hi = int(bounds[0]), int(bounds[-1])
    check_product(out[lo:hi], torch.float32, want[lo:hi].cpu(), err[lo:hi].cpu())
    assert (out[:lo] == 77).all() and (out[hi:] == 77).all()
