"""Infinities and NaN among an adapter's second weights: the value that the formula gives, not only where it goes."""
import math

import pytest
import torch

import moe_prefill_ffn_amd as mp
from test_lora import HALF, ids_of, reference
from test_mxfp4 import gen, strided

gpu = pytest.mark.gpu


def check_special(M, K, N, r, n, kind, base_type, out_type, dtype, whole, pad=0):
    g = gen(M + N + r)
    types = {"same": dtype, "f32": torch.float32}
    if whole:                                             # sums that 16 bits hold: their further parts are 0
        x, a = torch.randint(-2, 3, (M, K), generator=g).to(dtype), torch.randint(-1, 2, (n, r, K), generator=g).to(dtype)
        x[:, 6:], x[:, 0] = 0, 1.0
    else:
        x, a = torch.randn(M, K, generator=g).to(dtype), (torch.randn(n, r, K, generator=g) / math.sqrt(K)).to(dtype)
    x[M // 2] = 0.0                                       # sums of 0: NaN beside an infinity
    b = (torch.randn(n, N, r, generator=g) / math.sqrt(r)).to(dtype)
    for i in range(n):
        b[i, (3 * i) % N, r - 1] = math.inf
        b[i, (3 * i + 7) % N, i % r] = -math.inf
        b[i, N - 1 - i % N, :2] = torch.tensor([math.inf, -math.inf], dtype=dtype)
    b[n - 1, N // 2, r // 2] = math.nan
    scales = 0.5 + torch.rand(n, generator=g)
    base = torch.randn(M, N, generator=g).to(types[base_type]) if base_type else None
    ids = ids_of(kind, M, n, g)
    out, buf = strided(torch.zeros(M, N, dtype=types[out_type]), pad)
    bd = strided(base, pad)[0] if base_type else None
    mp.moe_lora_add(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), bd, out, scales=scales.cuda())
    want, err = reference(x, a, b.nan_to_num(0, 0, 0), ids, base, scales, types[out_type], dtype == torch.bfloat16)
    special = torch.zeros(M, N, dtype=torch.float64)
    for i in range(n):
        at = (ids == i).nonzero().flatten()
        s = torch.sign(x[at].double() @ a[i].double().t())
        for q in range(r):                                # products one by one: 0 times an infinity counts, times a number not
            odd = (~torch.isfinite(b[i, :, q])).nonzero().flatten()
            for c in odd.tolist():
                special[at, c] += s[:, q] * b[i, c, q].double()
    got = out.double().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(special))
    inf = torch.isinf(special)
    assert int(inf.sum()) > 0 or kind == "none" or M == 1
    assert torch.equal(got[inf], special[inf])
    fine = torch.isfinite(special)
    step = torch.finfo(types[out_type]).eps / 2
    tol = err + step * (want.abs() + err) + (2.0 ** -25 if types[out_type] == torch.float16 else 0.0)
    assert ((got - want).abs() <= tol)[fine].all()
    assert (buf[:, N:] == 77).all()


@gpu
@pytest.mark.parametrize("whole", [False, True])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("base_type,out_type", [("same", "same"), ("f32", "f32"), (None, "f32"), (None, "same"), ("f32", "same")])
@pytest.mark.parametrize("M,K,N,r,n,kind,pad", [
    (1, 512, 136, 16, 3, "one", 0), (2, 512, 135, 32, 2, "mixed", 1), (48, 200, 200, 24, 9, "wild", 0), (48, 200, 90, 24, 9, "mixed", 3),
    (600, 264, 152, 64, 7, "mixed", 0), (700, 128, 72, 128, 5, "runs", 0), (520, 96, 600, 200, 3, "mixed", 0),
    (1100, 264, 264, 16, 6, "mixed", 0), (1300, 200, 136, 40, 4, "runs", 8), (1030, 520, 72, 128, 3, "mixed", 0), (1025, 96, 200, 256, 3, "wild", 0)])
def test_values(M, K, N, r, n, kind, pad, base_type, out_type, dtype, whole):
    check_special(M, K, N, r, n, kind, base_type, out_type, dtype, whole, pad)
