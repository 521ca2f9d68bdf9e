"""Sums x A^T of one row over the whole range that products of fp16 numbers have: each counts with the bits that the header
promises, whatever the row's largest is."""
import math

import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref
from test_mxfp4 import gen, strided

gpu = pytest.mark.gpu


def bounded(x, a, b, ids, base, out_type):
    """(out, bound) in fp64.  s: K additions, and up to 24 of the parts' sums, each off by 2^-23 of the sum of magnitudes at most;
    of each s by itself 2^-22 is lost, or 2^-16 for an output of 16 bits.  s B^T: two products a rank and up to 7 windows' sums,
    2 r + 7 <= 3 r additions; a rounding of each window's factor and two of the term, one of the sum."""
    x, a, b = x.double(), a.double(), b.double()
    r, K = a.shape[1:]
    lost = 2.0 ** -22 if out_type == torch.float32 else 2.0 ** -16
    out = base.double().clone() if base is not None else torch.zeros(x.shape[0], b.shape[1], dtype=torch.float64)
    err = torch.zeros_like(out)
    for i in range(a.shape[0]):
        at = (ids == i).nonzero().flatten()
        s, es = x[at] @ a[i].t(), (K + 24) * 2.0 ** -23 * (x[at].abs() @ a[i].abs().t())
        es = es + lost * (s.abs() + es)
        delta = s @ b[i].t()
        ed = es @ b[i].abs().t() + 3 * r * 2.0 ** -23 * ((s.abs() + es) @ b[i].abs().t())
        out[at] += delta
        err[at] += ed + 3 * 2.0 ** -24 * (delta.abs() + ed)
    return out, err + 2.0 ** -24 * (out.abs() + err)


def wide(g, M, K, N, r, n, low):
    """Rank q's sums are of size 2^(16 - low q / (r - 1)) or so; columns that only the smaller ranks reach, columns that all
    reach with like products, and plain ones."""
    f16 = torch.float16
    x, a = torch.zeros(M, K), torch.zeros(n, r, K)
    half = K // 2
    x[:, :half], x[:, half:] = torch.randn(M, half, generator=g) * 2.0 ** 6, torch.randn(M, K - half, generator=g) * 2.0 ** -min(10.0, low / 4)
    e = 10 - low * torch.arange(r) / max(r - 1, 1)        # log2 of the sums' size
    big = e > -4                                          # of x's first half
    ea = torch.where(big, e - 6 - math.log2(half) / 2, e + min(10.0, low / 4) - math.log2(K - half) / 2).clamp(-22, 9)
    a[:, :, :half] = torch.randn(n, r, half, generator=g) * big[:, None]
    a[:, :, half:] = torch.randn(n, r, K - half, generator=g) * ~big[:, None]
    x, a = x.to(f16), (a * torch.exp2(ea)[:, None]).to(f16)
    b = torch.randn(n, N, r, generator=g)
    b[:, 0::3] *= torch.arange(r) >= r // 2               # 0 where the row's largest sums are
    b[:, 1::3] *= torch.exp2(-e.clamp(-14, 9))
    return x, a, b.to(f16)


SIZES = [(1, 64, 40, 8, 1, 36), (3, 264, 72, 16, 2, 20), (16, 128, 63, 32, 1, 44), (40, 72, 136, 24, 5, 36), (90, 64, 40, 256, 3, 44), (600, 200, 72, 64, 7, 28),
         (700, 520, 40, 128, 2, 44), (1100, 128, 136, 16, 3, 36), (1030, 64, 72, 64, 1, 44), (1500, 264, 40, 128, 6, 20), (1100, 72, 72, 256, 2, 44), (1200, 64, 72, 8, 1, 28)]


@gpu
@pytest.mark.parametrize("out_type", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("base_type", [None, torch.float32, torch.float16])
@pytest.mark.parametrize("M,K,N,r,n,low", SIZES)
def test_wide_rows(M, K, N, r, n, low, base_type, out_type):
    g = gen(M + r)
    x, a, b = wide(g, M, K, N, r, n, low)
    ids = torch.randint(0, n, (M,), generator=g).int()
    base = (torch.randn(M, N, generator=g) * 2.0 ** -20).to(base_type) if base_type else None
    out, buf = strided(torch.zeros(M, N, dtype=out_type), 8)
    mp.moe_lora_add(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), base.cuda() if base_type else None, out)
    want, err = bounded(x, a, b, ids, base, out_type)
    tol = err + ref.half_step(out_type) * (want.abs() + err) + ref.least_step(out_type)
    assert ((out.double().cpu() - want).abs() <= tol).all()
    assert (buf[:, N:] == 77).all()


@gpu
@pytest.mark.parametrize("M", [2, 50, 800, 1300])
def test_the_ends_of_the_range(M):
    """One rank's sum 2^-48, the smallest product that there is, beside one of 2^30 and a NaN-free infinity in the weights."""
    r, K, N = 16, 64, 72
    x, a, b = torch.zeros(M, K), torch.zeros(1, r, K), torch.zeros(1, N, r)
    x[:, 0], x[:, 1] = 2.0 ** 15, 2.0 ** -24
    a[0, 0, 0], a[0, 5, 1] = 2.0 ** 15, 2.0 ** -24
    a[0, 9, 1], a[0, 15, 1] = 3.0, -(2.0 ** -9)
    b[0, :, 5] = 1.0
    b[0, 8:, 9] = 2.0 ** -24
    b[0, 16:, 15] = 2.0 ** 8
    b[0, 24:, 0] = 1.0
    b[0, 32, 5], b[0, 33, 15], b[0, 34, 5], b[0, 34, 15] = math.inf, math.inf, math.inf, math.inf
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    out = mp.moe_lora_add(x.half().cuda(), a.half().cuda(), b.half().cuda(), ids, dtype=torch.float32).double().cpu()
    want = torch.full((N,), 2.0 ** -48, dtype=torch.float64)
    want[8:] += 3.0 * 2.0 ** -48
    want[16:] -= 2.0 ** -25
    want[24:] += 2.0 ** 30
    want[32], want[33], want[34] = math.inf, -math.inf, math.nan
    same = (out == want.float().double()) | (torch.isnan(out) & torch.isnan(want))
    assert same.all(), (~same).nonzero()[0].tolist()
