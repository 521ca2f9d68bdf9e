"""16-bit products of more tiles than a persistent workgroup lists at a time (256): every row of the result against the
formula, dense and over groups, whose bounds are scanned again for each further list."""
import math

import pytest
import torch

import moe_prefill_ffn_amd as mp
from test_experts16_limits import launches_of

gpu = pytest.mark.gpu
# M, N, K, groups (0: dense), rows of a tile
CASES = [(17_200_011, 32, 8, 0, 128), (16_900_000, 24, 128, 0, 128), (16_900_123, 250, 8, 0, 256), (17_300_000, 32, 8, 37, 128), (17_300_000, 40, 16, 1500, 128)]


def test_these_sizes_take_several_lists(tmp_path):
    for (M, N, K, G, rows), [(_, _, lds, grid, _, threads)] in zip(CASES, launches_of(tmp_path, [c[:4] + (0, 0) for c in CASES])):
        assert threads == 256 and M // rows > 256 * grid, (M, N, K, G, grid, lds)


def check_rows(out, a, b, src, group, swiglu):
    """In pieces; b [G, NB, K], group of each row or None."""
    M, K = out.shape[0], a.shape[1]
    step = (1 << 28) // (b.shape[1] * K if group is not None else 16 * b.shape[1])
    for i in range(0, M, step):
        x = a[src[i:i + step].long()].double() if src is not None else a[i:i + step].double()
        if group is None:
            z, mag = x @ b[0].double().t(), x.abs() @ b[0].double().abs().t()
        else:
            prod = x[:, None] * b[group[i:i + step]].double()
            z, mag = prod.sum(-1), prod.abs().sum(-1)
        err = K * 2.0 ** -23 * mag
        if swiglu:
            h = z.shape[1] // 2
            g, u, eg, eu = z[:, :h], z[:, h:], err[:, :h], err[:, h:]
            s = g * torch.sigmoid(g)
            z = s * u                                     # |silu'| <= 1.1; its evaluation 8 half steps
            err = 1.1 * eg * (u.abs() + eu) + s.abs() * eu + 8 * 2.0 ** -24 * z.abs()
        bad = (out[i:i + step].double() - z).abs() > err + 2.0 ** -8 * (z.abs() + err)
        assert not bad.any(), (i + bad.nonzero()[0]).tolist()


@gpu
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K,G", [c[:4] for c in CASES])
def test_every_row(M, N, K, G, swiglu):
    g = torch.Generator(device="cuda").manual_seed(M + G)
    NB = 2 * N if swiglu else N
    b = (torch.randn(max(G, 1), NB, K, generator=g, device="cuda") / math.sqrt(K)).bfloat16()
    bounds = rows = group = None
    A = M
    if G:
        A = 100_000
        cuts = torch.randint(0, M + 1, (G - 1,), generator=g, device="cuda").sort().values
        cuts[3:6] = cuts[3]                               # empty groups
        bounds = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), M)])
        rows = torch.randint(0, 2 * A, (M,), generator=g, device="cuda", dtype=torch.int32)
        group = torch.searchsorted(bounds[1:], torch.arange(M, device="cuda"), right=True)
    a = torch.randn(A, K, generator=g, device="cuda", dtype=torch.bfloat16)
    out = torch.full((M, N), 77.0, dtype=torch.bfloat16, device="cuda")
    mp.moe_grouped_gemm(a, b if G else b[0], out, bounds=bounds.int() if G else None, rows=rows, top_k=2 if G else 1, swiglu=swiglu)
    check_rows(out, a, b, rows // 2 if G else None, group, swiglu)
