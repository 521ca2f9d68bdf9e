"""Masked logits, wide routing and pool layers of the few-token layer in each of its kernels: pairs with the fused
down and combine, pairs without, chunks; every type; a workspace that holds NaN and -1."""
import math

import pytest
import torch

import moe_prefill_ffn_amd as mp
from test_decode import DTYPES, Layer, check, inputs, layers, run  # noqa: F401  (layers: a fixture)

gpu = pytest.mark.gpu


def dirty(L, T):
    return torch.full((mp.moe_decode_workspace_size(L.d, L.f, L.E, L.k, T),), 255, dtype=torch.uint8, device="cuda")


def check_masked(L, h, blob, x, lg):
    y, ex = run(L, h, x, lg, blob, workspace=dirty(L, x.shape[0]))
    check(y, ex, L, x, lg)
    for t in range(x.shape[0]):
        if (lg[t] == -math.inf).all():
            assert (y[t] == 0).all() and (ex["eidx"][t] == -1).all() and (ex["weights"][t] == 0).all()


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,T", [((2048, 768, 9, 8), 1), ((1024, 512, 9, 8), 1), ((1184, 1376, 5, 2), 2), ((1024, 64, 5, 2), 1), ((1024, 64, 5, 2), 4), ((1024, 96, 5, 1), 8),
                                     ((2048, 768, 9, 8), 3), ((96, 64, 5, 2), 3), ((2048, 768, 9, 8), 20), ((1024, 64, 5, 2), 80)])
def test_masks_in_every_kernel(layers, shape, T, dtype):
    L, h, blob = layers(*shape)
    E, k, low = L.E, L.k, torch.finfo(torch.float32).min
    g = torch.Generator().manual_seed(T)
    rows = [torch.full((E,), -math.inf), torch.full((E,), low), torch.randn(E, generator=g)]
    one = torch.full((E,), -math.inf)
    one[E - 1] = low                                      # one expert, at the type's lowest value
    rows.append(one)
    for live in (k - 1, k, k + 1):                        # fewer experts than slots, as many, one more
        r = torch.full((E,), -math.inf)
        at = torch.randperm(E, generator=g)[: max(0, min(E, live))]
        r[at] = torch.randn(at.numel(), generator=g)
        rows.append(r)
    for first in range(0, len(rows), T):
        lg = torch.stack([rows[(first + i) % len(rows)] for i in range(T)])
        x, _ = inputs(T, L, dtype, seed=first)
        x[(lg == -math.inf).all(1)] = math.nan            # an empty slot of a padded batch: whatever it holds
        if T > 1:
            xr = torch.where(torch.isnan(x), torch.zeros_like(x), x)
            y, ex = run(L, h, x, lg, blob, workspace=dirty(L, T))
            check(y, ex, L, xr, lg)
            assert (y[(lg == -math.inf).all(1)] == 0).all()
        elif torch.isnan(x).any():
            y, ex = run(L, h, x, lg, blob, workspace=dirty(L, T))
            assert (y == 0).all() and (ex["eidx"] == -1).all() and (ex["weights"] == 0).all()
        else:
            check_masked(L, h, blob, x, lg)


@gpu
@pytest.mark.parametrize("T", [1, 2, 40])
@pytest.mark.parametrize("E,k", [(64, 3), (65, 3), (128, 4), (129, 4), (200, 8), (256, 8), (257, 4), (300, 4), (1000, 3), (1024, 8)])
def test_routing_over_many_experts(layers, E, k, T):
    """Few pairs and many; equal logits in lanes and 64-expert groups that hold them together."""
    L, h, blob = layers(64, 32, E, k)
    x, lg = inputs(T, L, torch.float32, seed=E + T)
    check_masked(L, h, blob, x, lg)
    lg = torch.randint(0, 3, (T, E), generator=torch.Generator().manual_seed(E)).float()
    check_masked(L, h, blob, x, lg)
    lg[:] = -1.0
    lg[:, E - 1] = lg[:, E // 2] = lg[:, E - 1 - E // 4] = 2.0     # ties across the groups, the last expert among them
    check_masked(L, h, blob, x, lg)
    lg[:] = -math.inf
    lg[:, E - 1] = lg[:, E // 2] = 0.5
    check_masked(L, h, blob, x, lg)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("active_only", [False, True])
def test_pool_layers_of_real_width(dtype, active_only):
    """K is split over the waves here, otherwise by the pairs' kernels than by the chunks' that an active-only
    pool takes: both within the bound."""
    Ls = [Layer(1184, 352, 12, 4, seed=s) for s in range(3)]
    blobs = [L.host.clone().pin_memory() for L in Ls]
    h = mp.moe_prefill_create(1184, 352, 12, 4, 8)
    mp.stream_pool_configure(h, blobs, prefetch_depth=0 if active_only else 1, resident_layers=0, requested_slots=2, active_only=active_only)
    for _ in range(2):
        for i, L in enumerate(Ls):
            x, lg = inputs(2, L, dtype, seed=i)
            lg[0, 2:] = -math.inf                         # two of four slots without an expert
            y, ex = run(L, h, x, lg, None, layer=i, workspace=dirty(L, 2))
            check(y, ex, L, x, lg)
    st = mp.moe_prefill_get_stats(h)
    assert st["sparse_loads"] == (6 if active_only else 0)
    h.close()
