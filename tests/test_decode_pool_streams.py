"""Few-token calls of one handle on two streams, on layers of its pool: a slot is not filled again under a call that
still reads it on the other stream."""
import pytest
import torch

import moe_prefill_ffn_amd as mp
from test_decode import Layer, check, inputs

gpu = pytest.mark.gpu


def ready(T, **pool):
    Ls = [Layer(1184, 352, 12, 4, seed=s) for s in range(4)]
    h = mp.moe_prefill_create(1184, 352, 12, 4, 8)
    mp.stream_pool_configure(h, [L.host.clone().pin_memory() for L in Ls], **pool)
    x, lg = inputs(T, Ls[0], torch.float32, seed=3)
    return h, x.cuda(), lg.cuda(), lambda y, l: check(y.cpu(), None, Ls[l], x, lg)


@gpu
@pytest.mark.parametrize("T", [1, 3, 8])
@pytest.mark.parametrize("pool", [dict(prefetch_depth=1, requested_slots=2), dict(prefetch_depth=0, requested_slots=2),
                                  dict(prefetch_depth=0, requested_slots=2, active_only=True)])
def test_a_slow_stream_keeps_its_layer(T, pool):
    h, x, lg, check_y = ready(T, **pool)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for first in range(3):
        ys = torch.full_like(x, 77.0)
        outs = []
        torch.cuda.synchronize()
        with torch.cuda.stream(a):
            torch.cuda._sleep(20_000_000)
            mp.moe_decode_run_layer(h, x, lg, ys, layer=first)
        with torch.cuda.stream(b):
            for l in [first, *(l % 4 for l in range(first + 1, first + 5))]:   # the same layer, then the slots' turn
                y = torch.full_like(x, 77.0)
                mp.moe_decode_run_layer(h, x, lg, y, layer=l)
                outs.append((y, l))
        torch.cuda.synchronize()
        check_y(ys, first)
        for y, l in outs:
            check_y(y, l)
    h.close()


@gpu
def test_a_resident_layer_in_a_graph_and_eager_calls_around_it():
    h, x, lg, check_y = ready(3, prefetch_depth=1, resident_layers=3, requested_slots=4)
    y, ws = torch.empty_like(x), torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    run = lambda out, l: mp.moe_decode_run_layer(h, x, lg, out, layer=l, workspace=ws)  # noqa: E731
    eager = []
    for l in range(4):                                    # every layer is in its slot: nothing is copied under the capture
        run(y, l)
        torch.cuda.synchronize()
        check_y(y, l)
        eager.append(y.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(y, 0)
    for i in range(3):
        y.fill_(77.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[0])
        for l in range(4):
            run(y, l)
            torch.cuda.synchronize()
            assert torch.equal(y, eager[l])
    h.close()
