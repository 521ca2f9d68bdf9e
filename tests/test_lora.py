"""The low-rank adapters of many requests against a plain 64-bit form with a derived bound, alone and beside the
projections, and their refusals."""
import ctypes
import math

import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref
from test_mxfp4 import gen, strided

gpu = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]


# ----------------------------------------------------------- refusals (CPU) ---

def lora_args(**kw):
    a = mp.moe_lora_args_t()
    a.struct_size = ctypes.sizeof(a)
    a.x, a.a, a.b, a.adapters, a.scales, a.base, a.out = 4096, 8192, 16384, 32768, 65536, 131072, 262144    # never read
    a.x_stride = a.K = 64
    a.base_stride = a.out_stride = a.N = 40
    a.M, a.rank, a.n_adapters, a.dtype = 4, 16, 3, mp.MOE_BF16
    a.workspace, a.workspace_bytes = 524288, 1 << 30
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(struct_size=12), dict(dtype=mp.MOE_F32), dict(dtype=3), dict(out_dtype=3), dict(base_dtype=-1), dict(M=-1), dict(M=(1 << 23) + 1),
    dict(K=0), dict(K=60), dict(K=(1 << 20) + 8, x_stride=1 << 21), dict(rank=0), dict(rank=12), dict(rank=264), dict(N=0), dict(N=(1 << 20) + 1),
    dict(n_adapters=0), dict(n_adapters=(1 << 20) + 1), dict(x=None), dict(a=None), dict(b=None), dict(adapters=None), dict(out=None),
    dict(workspace=None), dict(workspace_bytes=255), dict(workspace=524289), dict(x_stride=56), dict(x_stride=68), dict(base_stride=39),
    dict(out_stride=39), dict(out_stride=1 << 41), dict(x=4104), dict(a=8200), dict(b=16392), dict(adapters=32770), dict(scales=65537),
    dict(base=131074), dict(out=262145)])
def test_refusals(bad):
    assert mp.lib().moe_lora_add(lora_args(**bad), None) == mp.MOE_EINVAL
    assert mp.moe_prefill_last_error()


def test_no_rows_is_a_no_op_without_pointers():
    a = lora_args(M=0, x=None, a=None, b=None, adapters=None, scales=None, base=None, out=None, workspace=None, workspace_bytes=0)
    assert mp.lib().moe_lora_add(a, None) == mp.MOE_OK
    assert mp.moe_lora_workspace_size(0, 64, 16) == 0


def test_workspace_holds_fewer_rows_too():
    for K in (8, 64, 1024, 4096, 1 << 20):
        sizes = [mp.moe_lora_workspace_size(M, K, 24) for M in range(0, 20000, 7)]
        assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
        assert sizes[-1] >= 4 * 24 * (20000 // 7 * 7)


@pytest.mark.parametrize("M,K,r", [(-1, 64, 16), (4, 63, 16), (4, 64, 4), (4, 64, 512), (1 << 24, 64, 16)])
def test_workspace_refusals(M, K, r):
    with pytest.raises(mp.MoePrefillError):
        mp.moe_lora_workspace_size(M, K, r)
    assert mp.lib().moe_lora_workspace_size(4, 64, 16, None) == mp.MOE_EINVAL


def test_binding_refuses_host_tensors():
    z = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        mp.moe_lora_add(z, z[None], z[None], torch.zeros(2, dtype=torch.int32))


# ------------------------------------------------------------------- values ---

def reference(x, a, b, adapters, base, scales, out_dtype, bf):
    """(out, bound on the kernel's distance) in fp64; bf: bf16 adapters, else fp16.

    s = x A^T: every of its K additions, and up to 24 of the parts' sums, is off by 2^-23 of the sum of magnitudes at
    most.  Its 16-bit parts lose 2^-16 of it for bf16 (2^-24 where three of them make an fp32 out), 2^-22 and 2^-39 of
    the row's largest for fp16.  s B^T: up to three products a rank, additions as above.  Then three roundings
    of the term and one of the sum, 2^-24 each."""
    M, N = x.shape[0], b.shape[1]
    K, r = x.shape[1], a.shape[1]
    dev = x.device
    x, a, b = x.double(), a.double(), b.double()
    out = base.double().clone() if base is not None else torch.zeros(M, N, dtype=torch.float64, device=dev)
    err = torch.zeros_like(out)
    lost = (2.0 ** -24 if out_dtype == torch.float32 else 2.0 ** -16) if bf else 2.0 ** -22
    floor = 0.0 if bf else 2.0 ** -39
    for i in range(a.shape[0]):
        at = (adapters == i).nonzero().flatten()
        if not at.numel():
            continue
        s, mag = x[at] @ a[i].t(), x[at].abs() @ a[i].abs().t()
        es = (K + 24) * 2.0 ** -23 * mag
        es = es + lost * (s.abs() + es) + floor * (s.abs() + es).amax(-1, keepdim=True)
        c = 1.0 if scales is None else float(scales[i])
        delta = c * (s @ b[i].t())
        ed = abs(c) * (es @ b[i].abs().t() + 3 * r * 2.0 ** -23 * ((s.abs() + es) @ b[i].abs().t()))
        out[at] += delta
        err[at] += ed + 3 * 2.0 ** -24 * (delta.abs() + ed)
    return out, err + 2.0 ** -24 * (out.abs() + err)


def check(out, x, a, b, adapters, base, scales):
    want, err = reference(x, a, b, adapters, base, scales, out.dtype, a.dtype == torch.bfloat16)
    got = out.double().to(want.device)
    tol = err + ref.half_step(out.dtype) * (want.abs() + err) + ref.least_step(out.dtype)
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float((got - want).abs().max()))


def ids_of(kind, M, n, g):
    """Adapters of M rows: one for all, runs of rows, each its own, none at all, some out of range."""
    if kind == "one":
        return torch.full((M,), n - 1).int()
    if kind == "none":
        return torch.full((M,), -1).int()
    if kind == "runs":
        return (torch.arange(M) * min(n, M) // M).int()
    ids = torch.randint(0, n, (M,), generator=g)
    if kind == "wild":
        ids = torch.where(torch.arange(M) % 3 == 1, torch.tensor([-1, n, (1 << 31) - 1, -(1 << 31)])[torch.arange(M) % 4], ids)
    return ids.int()


SHAPES = [(1, 8, 1, 8, 1), (1, 4096, 300, 16, 3), (2, 72, 64, 24, 2), (15, 264, 65, 8, 20), (16, 520, 257, 32, 5), (17, 1184, 130, 40, 40),
          (48, 200, 1027, 64, 30), (65, 1000, 96, 72, 7), (130, 128, 72, 128, 9), (300, 344, 260, 136, 12), (513, 96, 40, 256, 3),
          (700, 640, 513, 16, 8), (1500, 256, 200, 96, 5)]


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("base_type,out_type", [("same", "same"), ("f32", "f32"), ("f32", "same"), (None, "f32"), (None, "same")])
@pytest.mark.parametrize("M,K,N,r,n", SHAPES)
def test_lora(M, K, N, r, n, base_type, out_type, dtype):
    g = gen(M + K + N + r)
    types = {"same": dtype, "f32": torch.float32}
    x = torch.randn(M, K, generator=g).to(dtype)
    a = (torch.randn(n, r, K, generator=g) / math.sqrt(K)).to(dtype).cuda()
    b = (torch.randn(n, N, r, generator=g) / math.sqrt(r)).to(dtype).cuda()
    scales = 0.5 + torch.rand(n, generator=g)
    base = torch.randn(M, N, generator=g).to(types[base_type]) if base_type else None
    pad = 8 * (M % 2)
    xd, _ = strided(x, pad)
    bd = strided(base, pad)[0] if base_type else None
    out, buf = strided(torch.zeros(M, N, dtype=types[out_type]), pad + M % 3)
    for kind in ("one", "runs", "mixed", "wild", "none"):
        ids = ids_of(kind, M, n, g).cuda()
        out.fill_(77.0)
        mp.moe_lora_add(xd, a, b, ids, bd, out, scales=scales.cuda() if M != 16 else None)
        check(out, xd, a, b, ids, bd, scales if M != 16 else None)
        assert (buf[:, N:] == 77).all()
        if kind == "none":
            assert torch.equal(out, (bd if bd is not None else torch.zeros_like(out)).to(out.dtype))


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("base_type,out_type", [("same", "same"), ("f32", "f32"), ("f32", "same"), (None, "f32"), (None, "same"), ("same", "f32"), ("other", "other")])
@pytest.mark.parametrize("M,K,N,r,n", [(1025, 200, 136, 8, 4), (1300, 1000, 264, 16, 9), (1100, 72, 1000, 32, 30), (2050, 512, 72, 64, 5), (1200, 96, 400, 120, 3),
                                       (1030, 264, 328, 200, 7), (1100, 1304, 136, 256, 2)])
def test_many_rows(M, K, N, r, n, base_type, out_type, dtype):
    """The kernels of more than 1024 rows, for each count of ranks that they hold at once and each size of base and out."""
    g = gen(M + K + N + r)
    other = torch.float16 if dtype == torch.bfloat16 else torch.bfloat16
    types = {"same": dtype, "f32": torch.float32, "other": other}
    x = torch.randn(M, K, generator=g).to(dtype)
    a = (torch.randn(n, r, K, generator=g) / math.sqrt(K)).to(dtype).cuda()
    b = (torch.randn(n, N, r, generator=g) / math.sqrt(r)).to(dtype).cuda()
    scales = (0.5 + torch.rand(n, generator=g)).cuda()
    base = torch.randn(M, N, generator=g).to(types[base_type]) if base_type else None
    xd, _ = strided(x, 8)
    bd = strided(base, 8)[0] if base_type else None
    out, buf = strided(torch.zeros(M, N, dtype=types[out_type]), 8)
    for kind in ("runs", "mixed", "wild", "none"):
        ids = ids_of(kind, M, n, g).cuda()
        out.fill_(77.0)
        mp.moe_lora_add(xd, a, b, ids, bd, out, scales=scales)
        check(out, xd, a, b, ids, bd, scales)
        assert (buf[:, N:] == 77).all()
        if base_type == out_type:                         # in place: the same bits
            inner = bd.clone()
            mp.moe_lora_add(xd, a, b, ids, inner, inner, scales=scales)
            assert torch.equal(inner, out)


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M", [1, 40, 1000])
def test_in_place_and_by_default(M, dtype):
    g = gen(M)
    x, a, b = [torch.randn(*s, generator=g).to(dtype).cuda() / 8 for s in ((M, 256), (4, 16, 256), (4, 100, 16))]
    ids, base = torch.randint(-1, 4, (M,), generator=g).int().cuda(), torch.randn(M, 100, generator=g).to(dtype).cuda()
    want = mp.moe_lora_add(x, a, b, ids, base)
    assert want.dtype == dtype
    ws = torch.full((mp.moe_lora_workspace_size(M + 50, 256, 16),), 255, dtype=torch.uint8, device="cuda")    # NaN bytes
    assert mp.moe_lora_add(x, a, b, ids, base, base, workspace=ws) is base
    assert torch.equal(base, want)


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("size", [1e-30, 1e-6, 1e4, 1e30])
def test_far_from_one(size, dtype):
    """x A^T far outside the range of fp16, or where bf16 would end: the bound holds relative to it."""
    g = gen(9)
    M, K, N, r, n = 20, 128, 50, 24, 3
    # fp16 holds 6e-8 to 6e4: there both factors end at 1e-3 and 1e2
    lo, hi = (1e-3, 1e2) if dtype == torch.float16 else (0.0, math.inf)
    fx = min(max(size ** 0.5, lo), hi)
    fa = min(max(size / fx, lo), hi)
    x, a = (torch.randn(M, K, generator=g) * fx).to(dtype), (torch.randn(n, r, K, generator=g) * fa).to(dtype)
    b = torch.randn(n, N, r, generator=g).to(dtype)
    ids = torch.randint(0, n, (M,), generator=g).int()
    out = mp.moe_lora_add(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), dtype=torch.float32)
    check(out, x, a, b, ids, None, None)


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M", [12, 600])
def test_ranks_of_very_different_size(M, dtype):
    """One rank's sums 2^20 times another's, their weights the other way round: both count."""
    g = gen(3)
    K, N, r = 64, 33, 16
    e = torch.where(torch.arange(r) % 2 == 0, 2.0 ** 10, 2.0 ** -10)
    x = torch.randn(M, K, generator=g).to(dtype).cuda()
    a = (torch.randn(1, r, K, generator=g) * e[:, None]).to(dtype).cuda()
    b = (torch.randn(1, N, r, generator=g) / e).to(dtype).cuda()
    ids = torch.zeros(M, dtype=torch.int32, device="cuda")
    out = mp.moe_lora_add(x, a, b, ids, dtype=torch.float32)
    check(out, x, a, b, ids, None, None)
    full = (x.double() @ a[0].double().t()) @ b[0].double().t()
    # fp16's second part ends at 2^-39 of a row's largest sum, here 2^-19 of the small ones, uniform roundings of which leave
    # 2^-18.5 at most; all others are of 2^-23 and below
    assert float((out.double() - full).norm() / full.norm()) < (2.0 ** -20 if dtype == torch.bfloat16 else 2.0 ** -18)


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M", [48, 2000])
def test_infinities_and_nan_reach_their_rows_only(M, dtype):
    g = gen(M)
    K, N, r, n = 200, 90, 24, 5
    x, a, b = [torch.randn(*s, generator=g).to(dtype) for s in ((M, K), (n, r, K), (n, N, r))]
    x[7, K - 1], x[M - 1, 0] = math.nan, math.inf
    a[1, r - 1, K - 1], b[2, 5, r - 1], b[3, N - 1, 0] = math.inf, math.nan, -math.inf
    ids = (torch.arange(M) % 6 - 1).int()                 # -1 .. 4
    scales = torch.ones(n)
    scales[4] = 2.0
    base = torch.randn(M, N, generator=g)
    out = mp.moe_lora_add(x.cuda(), a.cuda(), b.cuda(), ids.cuda(), base.cuda(), scales=scales.cuda(), dtype=torch.float32).cpu()
    bad = (ids == 1)[:, None].expand(M, N).clone()
    bad[7] |= ids[7] >= 0
    bad[M - 1] |= ids[M - 1] >= 0
    bad[:, 5] |= ids == 2
    bad[:, N - 1] |= ids == 3
    assert not torch.isfinite(out[bad]).any() and torch.isfinite(out[~bad]).all()
    assert torch.equal(out[ids < 0], base[ids < 0])
    clean = torch.where(bad, 0.0, out)
    want, err = reference(x.nan_to_num(0, 0, 0), a.nan_to_num(0, 0, 0), b.nan_to_num(0, 0, 0), ids, base, scales, torch.float32,
                          dtype == torch.bfloat16)
    assert ((clean.double() - want).abs() <= err + 2.0 ** -24 * want.abs())[~bad].all()


@gpu
@pytest.mark.parametrize("M", [5, 300, 3000])
def test_in_a_replayed_graph_and_on_two_streams(M):
    g = gen(M)
    K, N, r, n = 512, 300, 32, 6
    x, a, b = [(torch.randn(*s, generator=g) / 8).bfloat16().cuda() for s in ((M, K), (n, r, K), (n, N, r))]
    base, ids = torch.randn(M, N, generator=g).bfloat16().cuda(), torch.randint(-1, n, (M,), generator=g).int().cuda()
    ws, out = torch.empty(mp.moe_lora_workspace_size(M, K, r), dtype=torch.uint8, device="cuda"), torch.empty_like(base)
    run = lambda o, w=None, s=None: mp.moe_lora_add(x, a, b, ids, base, o, workspace=w, stream=s)  # noqa: E731
    run(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, ws)
    for kind in ("runs", "mixed", "none", "one", "wild"):
        ids.copy_(ids_of(kind, M, n, g))
        x.copy_(torch.randn(M, K, generator=g) / 8)
        out.fill_(77.0)
        graph.replay()
        want = run(torch.full_like(out, 55.0))
        torch.cuda.synchronize()
        assert torch.equal(out, want), kind
    sides, outs = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(6):
        sides[i % 2].wait_stream(torch.cuda.current_stream())
        outs.append(run(torch.full_like(out, 77.0), None, sides[i % 2]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


@gpu
def test_far_offsets():
    """Adapters that span more than 2^32 bytes, and x and out whose rows do."""
    K, N, r, n = 32768, 64, 64, 1100                      # A: 4.6 GB
    a = torch.zeros(n, r, K, dtype=torch.bfloat16, device="cuda")
    b = torch.zeros(n, N, r, dtype=torch.bfloat16, device="cuda")
    g = gen(1)
    a[n - 1] = (torch.randn(r, K, generator=g) / 180).bfloat16().cuda()
    b[n - 1] = torch.randn(N, r, generator=g).bfloat16().cuda()
    M, stride = 70, 1 << 26
    x = torch.zeros((M - 1) * stride + K, dtype=torch.bfloat16, device="cuda").as_strided((M, K), (stride, 1))
    x.copy_(torch.randn(M, K, generator=g))
    out = torch.empty((M - 1) * stride + N, device="cuda").as_strided((M, N), (stride, 1))
    ids = torch.full((M,), n - 1, dtype=torch.int32, device="cuda")
    mp.moe_lora_add(x, a, b, ids, out=out)
    check(out, x, a[-1:], b[-1:], ids - (n - 1), None, None)


@gpu
@pytest.mark.parametrize("M", [6, 700])
def test_beside_the_projections(M):
    """On an MXFP4 projection's output, and in place on a 16-bit one's."""
    g = gen(M)
    K, N, r, n = 256, 320, 16, 4
    x = torch.randn(M, K, generator=g).bfloat16().cuda()
    w = (torch.randn(N, K, generator=g) / 16).bfloat16().cuda()
    a, b = (torch.randn(n, r, K, generator=g) / 16).bfloat16().cuda(), (torch.randn(n, N, r, generator=g) / 4).bfloat16().cuda()
    ids, scales = torch.randint(-1, n, (M,), generator=g).int().cuda(), torch.rand(n, generator=g).cuda()
    base = mp.moe_mxfp4_gemm(*mp.moe_mxfp4_quantize(x), *mp.moe_mxfp4_quantize(w))
    check(mp.moe_lora_add(x, a, b, ids, base, scales=scales, dtype=torch.bfloat16), x, a, b, ids, base, scales)
    y = mp.moe_grouped_gemm(x, w)
    before = y.clone()
    mp.moe_lora_add(x, a, b, ids, y, y, scales=scales)
    check(y, x, a, b, ids, before, scales)
    merged = torch.stack([x[t].double() @ (w.double() + (scales[i].double() * b[i].double() @ a[i].double() if i >= 0 else 0)).t()
                          for t, i in enumerate(ids.tolist())])
    # two roundings to bf16, of the projection and of the sum
    assert float((y.double() - merged).norm() / merged.norm()) < 2.0 ** -8


@gpu
@pytest.mark.parametrize("T", [3, 200, 1500])
def test_a_captured_layer_with_adapters(T):
    """Row table, gate/up, down, a shared expert whose second product carries adapters in place, the combine: one graph,
    replayed on other inputs, routings and adapters between eager calls, against the eager run bit for bit."""
    g = gen(T)
    d, f, E, k, n, r = 128, 192, 9, 3, 5, 16
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, eidx, w = torch.empty(T, d, **bf), torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    ids = torch.empty(T, dtype=torch.int32, device="cuda")
    gu, dn = [(torch.randn(E + 1, *s, generator=g) / 16).to(**bf) for s in ((2 * f, d), (d, f))]
    a, b = (torch.randn(n, r, f, generator=g) / 16).to(**bf), (torch.randn(n, d, r, generator=g) / 4).to(**bf)

    def layer():
        bounds, rows, pos = mp.moe_group_rows(eidx, E)
        h = mp.moe_grouped_gemm(x, gu[:E], bounds=bounds, rows=rows, top_k=k, swiglu=True)
        dm = mp.moe_grouped_gemm(h, dn[:E], bounds=bounds)
        hs = mp.moe_grouped_gemm(x, gu[E], swiglu=True)
        shared = mp.moe_grouped_gemm(hs, dn[E], dtype=torch.float32)
        mp.moe_lora_add(hs, a, b, ids, shared, shared)
        return mp.moe_combine_rows(dm, w, pos, base=shared)

    def fill():
        x.copy_(torch.randn(T, d, generator=g))
        eidx.copy_(torch.rand(T, E, generator=g).topk(k, -1).indices.int())
        eidx[T // 2] = -1
        w.copy_(torch.rand(T, k, generator=g))
        ids.copy_(torch.randint(-1, n, (T,), generator=g).int())

    fill()
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for _ in range(4):
        fill()
        y.fill_(77.0)
        graph.replay()
        want = layer()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@gpu
def test_binding_refusals_on_the_device():
    x, a, b = [torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((4, 64), (2, 16, 64), (2, 40, 16))]
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (lambda: mp.moe_lora_add(x, a[:, :, :32], b, ids), lambda: mp.moe_lora_add(x, a, b[:1], ids), lambda: mp.moe_lora_add(x, a[0], b, ids),
                lambda: mp.moe_lora_add(x, a, b, ids[:3]), lambda: mp.moe_lora_add(x, a, b, ids, torch.zeros(4, 39, device="cuda")),
                lambda: mp.moe_lora_add(x, a, b, ids, scales=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mp.moe_lora_add(x.float(), a, b, ids), lambda: mp.moe_lora_add(x, a.half(), b, ids), lambda: mp.moe_lora_add(x, a, b, ids.long()),
                lambda: mp.moe_lora_add(x, a.transpose(0, 1).contiguous().transpose(0, 1), b, ids), lambda: mp.moe_lora_add(x, a, b, ids.cpu()),
                lambda: mp.moe_lora_add(x, a, b, ids, dtype=torch.float64)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(mp.MoePrefillError):
        mp.moe_lora_add(x, a, b, ids, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(mp.MoePrefillError):
        mp.moe_lora_add(x[:, :60], a[:, :, :60].contiguous(), b, ids)
    assert mp.moe_lora_add(x[:0], a, b, ids[:0]).shape == (0, 40)
