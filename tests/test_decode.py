"""The MoE layer for a few tokens (moe_decode_run_layer) against the layer's formulas in 64 bits,
within bounds derived from its arithmetic; masks, padded batches, strides, pools, graphs, refusals."""
import math

import numpy as np
import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref

gpu = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


class Layer:
    """Seeded canonical weights and their packed blob."""

    def __init__(self, d, f, E, k, seed=0):
        self.d, self.f, self.E, self.k = d, f, E, k
        g = torch.Generator().manual_seed(seed * 1000 + d + f + E)
        q = lambda *s: torch.randint(-8, 8, s, generator=g, dtype=torch.int8)  # noqa: E731
        s = lambda n, i: ((0.5 + torch.rand(E, n, i // 32, generator=g)) / math.sqrt(i)).half()  # noqa: E731
        self.gu_q, self.gu_s, self.d_q, self.d_s = q(E, 2 * f, d), s(2 * f, d), q(E, d, f), s(d, f)

        class W:
            pass

        def expert(e):
            w = W()
            bits = lambda t: t[e].contiguous().numpy().view(np.uint16)  # noqa: E731
            w.wgu_q, w.wgu_s, w.wd_q, w.wd_s = self.gu_q[e].numpy(), bits(self.gu_s), self.d_q[e].numpy(), bits(self.d_s)
            return w

        self.host = torch.empty(mp.moe_prefill_layer_bytes(d, f, E), dtype=torch.uint8)
        mp.pack_layer(d, f, E, expert, self.host)

    def reference(self, x, logits):
        return ref.layer(x, logits, self.k, self.gu_q, self.gu_s, self.d_q, self.d_s)


def run(L, h, x, logits, blob, pad=0, exports=True, **kw):
    """x, logits on the CPU -> y and the exports, rows of x, logits and y in wider buffers."""
    T, d = x.shape
    wide = lambda t, p: torch.cat([t, torch.full((T, p), 77.0, dtype=t.dtype)], 1).cuda()  # noqa: E731
    xb, lb = wide(x, pad), wide(logits, pad)
    yb = torch.full((T, d + pad), 77.0, dtype=x.dtype, device="cuda")
    ex = dict(eidx=torch.full((T, L.k), -9, dtype=torch.int32, device="cuda"),
              weights=torch.full((T, L.k), -9.0, device="cuda")) if exports else None
    mp.moe_decode_run_layer(h, xb[:, :d], lb[:, : L.E], yb[:, :d], weights=blob, exports=ex, **kw)
    torch.cuda.synchronize()
    assert (yb[:, d:] == 77).all()
    return yb[:, :d].cpu(), ({n: t.cpu() for n, t in ex.items()} if ex else None)


def check(y, ex, L, x, logits):
    want, bound, eidx, wts = L.reference(x, logits)
    tol = bound + ref.half_step(x.dtype) * (want.abs() + bound) + ref.least_step(x.dtype)
    got = y.double()
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float((got - want).abs().max()))
    # the fixed-point steps average out over a row: 2^-23 (2^-15) of a block's largest, a few times its rms
    fixed = 2e-6 if x.dtype == torch.float32 else 2.0 ** -14
    assert float((got - want).norm()) <= (fixed + 1.2 * ref.half_step(x.dtype)) * float(want.norm()) + ref.least_step(x.dtype) * got.numel() ** 0.5
    if ex is not None:
        assert torch.equal(ex["eidx"], eidx)
        assert ((ex["weights"].double() - wts).abs() <= (2 * L.k + 8) * 2.0 ** -24 * wts + 1e-30).all()


def inputs(T, L, dtype, seed=1, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(T, L.d, generator=g)).to(dtype), torch.randn(T, L.E, generator=g)


@pytest.fixture(scope="module")
def layers():
    made = {}

    def get(d, f, E, k):
        if (d, f, E, k) not in made:
            L = Layer(d, f, E, k)
            made[d, f, E, k] = (L, mp.moe_prefill_create(d, f, E, k, 4), L.host.cuda())
        return made[d, f, E, k]

    yield get
    for _, h, _ in made.values():
        h.close()


# ----------------------------------------------------------- refusals (CPU) ---

def test_workspace_size_and_its_refusals():
    a = mp.moe_decode_workspace_size(2048, 768, 128, 8, 1)
    assert 0 < a < mp.moe_decode_workspace_size(2048, 768, 128, 8, 128)
    for bad in [(2048, 768, 128, 8, 129), (100, 768, 8, 2, 1), (64, 64, 8, 9, 1), (64, 64, 8, 2, 0), (64, 64, 1025, 2, 1)]:
        with pytest.raises(mp.MoePrefillError) as ei:
            mp.moe_decode_workspace_size(*bad)
        assert ei.value.code == mp.MOE_EINVAL


def test_null_handle_is_refused():
    assert mp.lib().moe_decode_run_layer(None, mp.moe_decode_io_t(), None) == mp.MOE_EINVAL


# ------------------------------------------------------------------- values ---

SHAPES = [(32, 32, 1, 1), (64, 96, 4, 4), (96, 64, 5, 2), (224, 160, 3, 2), (1184, 352, 12, 4), (2048, 768, 9, 8), (512, 1536, 6, 3)]


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("T", [1, 2, 9])
def test_layer(layers, shape, T, dtype):
    L, h, blob = layers(*shape)
    x, lg = inputs(T, L, dtype, seed=T)
    y, ex = run(L, h, x, lg, blob, pad=8 * (T - 1))
    check(y, ex, L, x, lg)


@gpu
@pytest.mark.parametrize("T,shape", [(40, (64, 64, 2, 1)), (1024, (64, 32, 3, 1)), (16, (64, 64, 64, 64)), (1, (32, 64, 1024, 300)),
                                     (17, (96, 32, 300, 60)), (128, (64, 96, 16, 8))])
def test_many_rows_and_many_experts(layers, T, shape):
    L, h, blob = layers(*shape)
    x, lg = inputs(T, L, torch.float32, seed=T)
    y, ex = run(L, h, x, lg, blob)
    check(y, ex, L, x, lg)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,shape", [(40, (64, 96, 4, 4)), (66, (96, 64, 5, 2)), (70, (224, 160, 3, 2)), (33, (1184, 352, 12, 4)), (17, (2048, 768, 9, 8)),
                                     (140, (32, 32, 1, 1))])
def test_more_than_128_pairs(layers, T, shape, dtype):
    L, h, blob = layers(*shape)
    x, lg = inputs(T, L, dtype, seed=T)
    y, ex = run(L, h, x, lg, blob, pad=16)
    check(y, ex, L, x, lg)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [3, 5])
def test_wide_experts_shared_by_few_tokens(layers, T, dtype):
    """Experts of 28 MB, 2 of 3 a token: read again for every token, or once for all."""
    L, h, blob = layers(4096, 4096, 3, 2)
    x, lg = inputs(T, L, dtype, seed=T)
    y, ex = run(L, h, x, lg, blob)
    check(y, ex, L, x, lg)


@gpu
@pytest.mark.parametrize("T", [1, 3, 8, 72])
def test_masks_ties_and_extreme_logits(layers, T):
    L, h, blob = layers(96, 64, 5, 2)
    low = torch.finfo(torch.float32).min
    cases = [[-math.inf] * 5, [-math.inf, -math.inf, 3.0, -math.inf, -math.inf], [0.0, -0.0, 0.0, -0.0, 0.0], [low] * 5,
             [low, -math.inf, low, -math.inf, 1.0], [-math.inf, 1.0, 1.0, 1.0, -math.inf], [88.0, -88.0, 3e38, -3e38, 0.0],
             [5.0, 5.0 - 1e-6, 1.0, 5.0, 2.0]]
    for first in range(0, len(cases), T):
        lg = torch.tensor([cases[(first + i) % len(cases)] for i in range(T)])
        x, _ = inputs(T, L, torch.float32, seed=first)
        y, ex = run(L, h, x, lg, blob)
        check(y, ex, L, x, lg)
        for t in range(T):
            if (lg[t] == -math.inf).all():
                assert (y[t] == 0).all() and (ex["eidx"][t] == -1).all() and (ex["weights"][t] == 0).all()


@gpu
@pytest.mark.parametrize("T", [5, 80])
def test_infinities_and_nan_stay_in_their_token(layers, T):
    L, h, blob = layers(96, 64, 5, 2)
    x, lg = inputs(T, L, torch.float32)
    clean, _ = run(L, h, x, lg, blob)
    x2, lg2 = x.clone(), lg.clone()
    x2[1, 3], x2[3, 95] = math.nan, math.inf
    lg2[4] = -math.inf
    x2[4] = math.nan                                      # an empty slot of a padded batch: whatever it holds
    y, _ = run(L, h, x2, lg2, blob)
    assert torch.isnan(y[[1, 3]]).all()
    assert torch.equal(y[[0, 2]], clean[[0, 2]]) and torch.equal(y[5:], clean[5:])
    assert (y[4] == 0).all()


@gpu
@pytest.mark.parametrize("scale", [1e-38, 1e-20, 1e15])
def test_range_of_the_activations(layers, scale):
    """Tiny blocks lose bits below 2^-126 of the fixed-point scale: the bound gains that absolute error."""
    L, h, blob = layers(224, 160, 3, 2)
    x, lg = inputs(3, L, torch.float32, scale=scale)
    y, ex = run(L, h, x, lg, blob)
    want, bound, _, _ = L.reference(x, lg)
    # h is of the second order in a small x and leaves fp32's range below scale^2 ~ 1e-38: absolute 2^-126 per term
    tol = bound + 2.0 ** -24 * want.abs() + 2.0 ** -126 * 8 * (L.d + L.f)
    assert ((y.double() - want).abs() <= tol).all()


@gpu
def test_a_block_of_mixed_magnitudes(layers):
    """One large value in a block of small ones: the error is relative to the block's largest."""
    L, h, blob = layers(64, 96, 4, 4)
    x, lg = inputs(4, L, torch.float32)
    x[:, 7] *= 1e4
    x[0, 40] = 0.0
    x[1] = 0.0
    y, ex = run(L, h, x, lg, blob)
    check(y, ex, L, x, lg)
    assert (y[1] == 0).all()


@gpu
@pytest.mark.parametrize("T", [1, 6, 30])
def test_y_may_be_x_and_runs_repeat_bit_for_bit(layers, T):
    L, h, blob = layers(2048, 768, 9, 8)
    x, lg = inputs(T, L, torch.bfloat16)
    y, _ = run(L, h, x, lg, blob)
    for _ in range(3):
        xd = x.cuda()
        mp.moe_decode_run_layer(h, xd, lg.cuda(), xd, weights=blob)
        assert torch.equal(xd.cpu(), y)


@gpu
def test_no_tokens(layers):
    L, h, blob = layers(64, 96, 4, 4)
    z = torch.empty(0, 64, device="cuda")
    mp.moe_decode_run_layer(h, z, torch.empty(0, 4, device="cuda"), z, weights=blob)


# ------------------------------------------------------ next to the framework ---

@gpu
def test_next_to_the_prompt_path(layers):
    """A prompt through run_layer, then its tokens again through the few-token layer: the same experts,
    and outputs apart by the prompt path's 8-bit rounding of x and h (half a step of 1/127 of a block's
    largest value each)."""
    L, _, blob = layers(2048, 768, 9, 8)
    h = mp.moe_prefill_create(L.d, L.f, L.E, L.k, 64)
    x, lg = inputs(64, L, torch.float32, seed=3)
    xd, lgd = x.cuda(), lg.cuda()
    y1, y2 = torch.empty_like(xd), torch.empty_like(xd)
    e1, e2 = (torch.empty(64, L.k, dtype=torch.int32, device="cuda") for _ in range(2))
    mp.moe_prefill_run_layer(h, xd, lgd, y1, weights=blob, exports={"eidx": e1})
    for t in range(0, 64, 16):
        mp.moe_decode_run_layer(h, xd[t:t + 16], lgd[t:t + 16], y2[t:t + 16], weights=blob, exports={"eidx": e2[t:t + 16]})
    torch.cuda.synchronize()
    h.close()
    assert torch.equal(e1, e2)
    # N(0,1) blocks of 32: largest ~ 2.5, rms error of a code = 2.5 / 127 / sqrt(12) = 0.6% of the rms, for x
    # (gate and up) and again, of a heavier-tailed product, for h: a few percent together
    assert float((y1 - y2).norm() / y1.norm()) < 0.04


@gpu
@pytest.mark.parametrize("active_only", [False, True])
def test_pool_layers_equal_resident_ones(active_only):
    Ls = [Layer(64, 96, 6, 2, seed=s) for s in range(4)]
    blobs = [L.host.clone().pin_memory() for L in Ls]
    h = mp.moe_prefill_create(64, 96, 6, 2, 8)
    want = []
    for L in Ls:
        x, lg = inputs(3, L, torch.float32, seed=8)
        want.append(run(L, h, x, lg, L.host.cuda())[0])
    mp.stream_pool_configure(h, blobs, prefetch_depth=0 if active_only else 1, resident_layers=0 if active_only else 1,
                             requested_slots=2, active_only=active_only)
    for _ in range(3):
        for i, L in enumerate(Ls):
            x, lg = inputs(3, L, torch.float32, seed=8)
            y, _ = run(L, h, x, lg, None, layer=i)
            assert torch.equal(y, want[i]), i
    # the prompt path and the few-token path take turns on one pool
    x, lg = inputs(3, Ls[2], torch.float32, seed=8)
    yp = torch.empty(3, 64, device="cuda")
    mp.moe_prefill_run_layer(h, x.cuda(), lg.cuda(), yp, layer=2)
    y, _ = run(Ls[3], h, x, lg, None, layer=3)
    assert torch.equal(y, want[3])
    st = mp.moe_prefill_get_stats(h)
    assert st["sparse_loads"] > 0 if active_only else st["prefetch_activated"] > 0
    h.close()


@gpu
def test_graphs_with_their_own_workspaces_and_an_eager_call_between(layers):
    L, h, blob = layers(1184, 352, 12, 4)
    T = (1, 7, 50)
    xs = [torch.empty(t, L.d, device="cuda") for t in T]
    ls = [torch.empty(t, L.E, device="cuda") for t in T]
    ys = [torch.empty(t, L.d, device="cuda") for t in T]
    graphs = []
    for x, l, y in zip(xs, ls, ys):
        x.normal_()
        l.normal_()
        ws = torch.empty(mp.moe_decode_workspace_size(L.d, L.f, L.E, L.k, x.shape[0]), dtype=torch.uint8, device="cuda")
        mp.moe_decode_run_layer(h, x, l, y, weights=blob, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mp.moe_decode_run_layer(h, x, l, y, weights=blob, workspace=ws)
        graphs.append((g, ws))
    gen = torch.Generator().manual_seed(4)
    for i in range(4):
        for x, l in zip(xs, ls):
            x.copy_(torch.randn(x.shape, generator=gen))
            l.copy_(torch.randn(l.shape, generator=gen))
        for ws in (w for _, w in graphs):
            ws.fill_(255)                                 # what a workspace holds does not matter
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in T]
        for (g, _), s in zip(graphs, streams):            # all at once, on streams of their own
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for x, l, y in zip(xs, ls, ys):
            e = torch.empty_like(y)
            mp.moe_decode_run_layer(h, x, l, e, weights=blob)
            torch.cuda.synchronize()
            assert torch.equal(e, y), i


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d,f", [(1, 16384, 32), (1, 32, 16384), (7, 16384, 32), (7, 32, 16384), (129, 16384, 32), (129, 32, 16384), (2, 16384, 1024)])
def test_longest_rows(layers, T, d, f, dtype):
    L, h, blob = layers(d, f, 2, 1)
    x, lg = inputs(T, L, dtype, seed=T)
    y, ex = run(L, h, x, lg, blob)
    check(y, ex, L, x, lg)


@gpu
def test_calls_at_once_on_two_streams(layers):
    """One handle, a workspace per call: the calls of each path (few pairs, chunks) run into each other."""
    L, h, blob = layers(2048, 768, 9, 8)
    calls = []
    for T in (1, 5, 16, 100):
        x, lg = (t.cuda() for t in inputs(T, L, torch.bfloat16, seed=T))
        want = torch.empty_like(x)
        mp.moe_decode_run_layer(h, x, lg, want, weights=blob)
        calls.append((x, lg, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    outs = []
    for _ in range(5):
        for (x, lg, want), s in zip(calls, streams):
            y = torch.full_like(want, 77.0)
            s.wait_stream(torch.cuda.current_stream())
            y.record_stream(s)
            mp.moe_decode_run_layer(h, x, lg, y, weights=blob, stream=s)
            outs.append((y, want))
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for y, w in outs)


@gpu
def test_on_another_stream_than_the_current_one(layers):
    L, h, blob = layers(2048, 768, 9, 8)
    x, lg = inputs(4, L, torch.float16)
    want, _ = run(L, h, x, lg, blob)
    xd, ld = x.cuda(), lg.cuda()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    for _ in range(8):                                    # workspaces of the allocator, reused between calls
        y = torch.empty_like(xd)
        y.record_stream(s)
        mp.moe_decode_run_layer(h, xd, ld, y, weights=blob, stream=s)
        torch.empty(1 << 20, device="cuda").fill_(1.0)
        outs.append(y)
    torch.cuda.synchronize()
    assert all(torch.equal(o.cpu(), want) for o in outs)


@gpu
def test_refusals_on_the_device(layers):
    L, h, blob = layers(64, 96, 4, 4)
    x, l, y = torch.zeros(2, 64, device="cuda"), torch.zeros(2, 4, device="cuda"), torch.full((2, 64), 77.0, device="cuda")
    call = lambda **kw: mp.moe_decode_run_layer(h, **{**dict(x=x, logits=l, y=y, weights=blob), **kw})  # noqa: E731
    big = torch.zeros(257, 64, device="cuda")
    for kw, err in [
            (dict(x=x.cpu()), TypeError), (dict(y=y.bfloat16()), TypeError), (dict(logits=l.double()), TypeError),
            (dict(x=x.double(), y=y.double()), TypeError), (dict(x=x[:1]), ValueError), (dict(y=y[:, :32]), ValueError),
            (dict(logits=l[:, :3]), ValueError), (dict(weights=None), ValueError), (dict(weights=blob[:-1]), ValueError),
            (dict(weights=blob.cpu()), TypeError), (dict(x=torch.zeros(64, 2, device="cuda").t()), ValueError),
            (dict(y=y[:1].expand(2, 64)), ValueError), (dict(exports={"gu": x}), KeyError),
            (dict(exports={"eidx": torch.zeros(7, dtype=torch.int32, device="cuda")}), ValueError),
            (dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), mp.MoePrefillError),
            (dict(x=big, y=big.clone(), logits=torch.zeros(257, 4, device="cuda")), mp.MoePrefillError),
            (dict(layer=0), mp.MoePrefillError),
            (dict(x=torch.zeros(130, device="cuda")[2:].view(2, 64)), mp.MoePrefillError)]:
        with pytest.raises(err):
            call(**kw)
    ws = torch.empty(mp.moe_decode_workspace_size(64, 96, 4, 4, 2) + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(mp.MoePrefillError):
        call(workspace=ws[8:])
    torch.cuda.synchronize()
    assert (y == 77).all()
