"""The operators of 16-bit experts -- row table, grouped product, combine -- against plain 64-bit
forms, at the sizes, masks and values where they can go wrong, alone and together, and their refusals."""
import ctypes
import math

import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref
from test_mxfp4 import check_product, gen, groups_of, strided

gpu = pytest.mark.gpu
HALF = [torch.bfloat16, torch.float16]
ALL = [torch.float32] + HALF


# ----------------------------------------------------------- refusals (CPU) ---

def group_args(**kw):
    a = mp.moe_group_args_t()
    a.struct_size = ctypes.sizeof(a)
    a.eidx, a.bounds, a.rows, a.pos = 4096, 8192, 16384, 32768      # never read: every case below is refused first
    a.n_pairs, a.n_groups = 16, 4
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(struct_size=4), dict(n_pairs=-1), dict(n_pairs=(1 << 27) + 1), dict(n_groups=0), dict(n_groups=1025), dict(eidx=None),
    dict(bounds=None), dict(eidx=4098), dict(bounds=8193), dict(rows=16386), dict(pos=32769), dict(counts=130),
    dict(n_pairs=5000), dict(n_pairs=5000, workspace=65536, workspace_bytes=31), dict(n_pairs=5000, workspace=65600, workspace_bytes=1 << 20)])
def test_group_refusals(bad):
    assert mp.lib().moe_group_rows(group_args(**bad), None) == mp.MOE_EINVAL
    assert "group" in mp.moe_prefill_last_error() or "struct_size" in mp.moe_prefill_last_error()


@pytest.mark.parametrize("P,E", [(-1, 4), (1 << 28, 4), (10, 0), (10, 1025)])
def test_group_workspace_refusals(P, E):
    with pytest.raises(mp.MoePrefillError):
        mp.moe_group_workspace_size(P, E)
    assert mp.lib().moe_group_workspace_size(10, 4, None) == mp.MOE_EINVAL


def test_group_workspace_size():
    assert mp.moe_group_workspace_size(0, 1) == mp.moe_group_workspace_size(4096, 1024) == 0
    for P in (4097, 65536, 300001, 1 << 27):              # a count a group and workgroup, at most 256 of them
        for E in (1, 60, 1024):
            assert 4 * E <= mp.moe_group_workspace_size(P, E) <= 256 * 4 * E + 255


def gemm_args(**kw):
    a = mp.moe_grouped_gemm_args_t()
    a.struct_size = ctypes.sizeof(a)
    a.a, a.b, a.out = 4096, 8192, 65536
    a.a_rows, a.n_groups, a.top_k, a.M, a.N, a.K, a.a_stride, a.b_stride, a.out_stride = 4, 1, 1, 4, 8, 64, 64, 64, 8
    a.dtype = a.out_dtype = mp.MOE_BF16
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(struct_size=0), dict(dtype=mp.MOE_F32), dict(dtype=3), dict(out_dtype=mp.MOE_F16), dict(out_dtype=-1), dict(swiglu=2),
    dict(K=0), dict(K=12), dict(K=(1 << 20) + 8, a_stride=1 << 21, b_stride=1 << 21), dict(N=0), dict(N=1 << 21), dict(M=-1),
    dict(M=(1 << 27) + 1, a_rows=1 << 28), dict(M=1 << 24, a_rows=1 << 24, N=1 << 20, out_stride=1 << 20),
    dict(a_rows=1 << 31), dict(n_groups=0), dict(n_groups=2), dict(n_groups=65536, bounds=128), dict(top_k=0),
    dict(a=None), dict(b=None), dict(out=None), dict(a_rows=0), dict(a_rows=3), dict(a_rows=1, top_k=3), dict(a_rows=0, rows=128),
    dict(a_stride=56), dict(b_stride=56), dict(out_stride=7), dict(a_stride=68), dict(b_stride=1 << 41), dict(b_stride=65),
    dict(n_groups=2, bounds=128, b_group_stride=-64), dict(n_groups=2, bounds=128, b_group_stride=516),
    dict(a=4104), dict(b=8200), dict(out=65537), dict(out=65538, out_dtype=mp.MOE_F32), dict(bounds=130), dict(rows=129)])
def test_gemm_refusals(bad):
    assert mp.lib().moe_grouped_gemm(gemm_args(**bad), None) == mp.MOE_EINVAL
    assert mp.moe_prefill_last_error()


def combine_args(**kw):
    a = mp.moe_combine_args_t()
    a.struct_size = ctypes.sizeof(a)
    a.d, a.weights, a.pos, a.base, a.y = 4096, 8192, 16384, 32768, 65536
    a.d_stride = a.base_stride = a.y_stride = a.N = 64
    a.d_rows, a.n_tokens, a.top_k = 8, 4, 2
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(struct_size=8), dict(d_dtype=3), dict(base_dtype=-1), dict(y_dtype=9), dict(N=0), dict(N=(1 << 20) + 1), dict(top_k=0),
    dict(top_k=1025), dict(n_tokens=-1), dict(n_tokens=(1 << 23) + 1), dict(d_rows=-1), dict(d_rows=1 << 31), dict(d=None),
    dict(weights=None), dict(pos=None), dict(y=None), dict(d_stride=63), dict(base_stride=63), dict(y_stride=-64), dict(y_stride=1 << 41),
    dict(d=4098), dict(base=32769, base_dtype=mp.MOE_F16), dict(y=65538), dict(weights=8194), dict(pos=16385)])
def test_combine_refusals(bad):
    assert mp.lib().moe_combine_rows(combine_args(**bad), None) == mp.MOE_EINVAL
    assert mp.moe_prefill_last_error()


def test_calls_of_no_rows_are_no_ops_without_pointers():
    assert mp.lib().moe_grouped_gemm(gemm_args(M=0, a=None, b=None, out=None, a_rows=0), None) == mp.MOE_OK
    assert mp.lib().moe_combine_rows(combine_args(n_tokens=0, d=None, weights=None, pos=None, base=None, y=None), None) == mp.MOE_OK


def test_binding_refuses_host_tensors():
    z, i = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, dtype=torch.int32)
    with pytest.raises(TypeError):
        mp.moe_group_rows(i, 4)
    with pytest.raises(TypeError):
        mp.moe_grouped_gemm(z, z)
    with pytest.raises(TypeError):
        mp.moe_combine_rows(z, torch.zeros(2, 2), i)


# -------------------------------------------------------------------- group ---

def table(eidx, E):
    """Bounds, rows in group order, pos and counts, one pair after the other."""
    lists = [[] for _ in range(E)]
    flat = eidx.flatten().tolist()
    for p, e in enumerate(flat):
        if 0 <= e < E:
            lists[e].append(p)
    pos, rows, bounds = [-1] * len(flat), [], [0]
    for members in lists:
        for p in members:
            pos[p] = len(rows)
            rows.append(p)
        bounds.append(len(rows))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(bounds), i32(rows), i32(pos).view(eidx.shape), i32([len(m) for m in lists])


def check_table(eidx, E, **kw):
    P = eidx.numel()
    dev = eidx.cuda()
    rows = torch.full((P + 8,), -77, dtype=torch.int32, device="cuda")
    counts = torch.full((E,), -77, dtype=torch.int32, device="cuda")
    pos = dev if kw.get("in_place") else None
    bounds, got_rows, pos = mp.moe_group_rows(dev, E, rows=rows[:P], counts=counts, pos=pos)
    want = table(eidx, E)
    n = int(want[0][-1])
    assert torch.equal(bounds.cpu(), want[0]) and torch.equal(pos.cpu(), want[2]) and torch.equal(counts.cpu(), want[3])
    assert torch.equal(rows[:n].cpu(), want[1]) and (rows[n:] == -77).all()


@gpu
@pytest.mark.parametrize("E", [1, 2, 60, 64, 256, 1023, 1024])
@pytest.mark.parametrize("P", [0, 1, 63, 64, 65, 192, 1000, 4095, 4096, 4097, 5121, 70001])
def test_group(P, E):
    g = gen(P + E)
    check_table(torch.randint(-1, E, (P,), generator=g).int(), E)
    skew = (E * torch.rand(P, generator=g) ** 3).int()    # most in the first groups
    check_table(skew, E, in_place=True)


@gpu
@pytest.mark.parametrize("P", [70, 4096, 9000])
def test_group_masks_and_unsound_ids(P):
    for eidx in (torch.full((P,), -1), torch.full((P,), 5), torch.full((P,), 9), torch.arange(P) % 10, torch.arange(P).flip(0) // (P // 10 + 1)):
        check_table(eidx.int(), 10)
    i = torch.arange(P)
    wild = torch.where(i % 3 == 0, i % 10, torch.where(i % 3 == 1, torch.tensor(-(1 << 31)), torch.tensor((1 << 31) - 1)))
    check_table(wild.int(), 10)
    check_table(torch.where(i % 2 == 0, 10, 9).int(), 10)


@gpu
def test_group_of_more_pairs_than_one_round_of_workgroups():
    g = gen(3)
    eidx = torch.randint(0, 300, (400001,), generator=g).int()
    bounds, rows, pos = mp.moe_group_rows(eidx.cuda(), 300)
    order = torch.sort(eidx, stable=True)
    assert torch.equal(rows.cpu().long(), order.indices)
    assert torch.equal(bounds.cpu().long(), torch.searchsorted(order.values, torch.arange(301).int()))
    assert torch.equal(pos.cpu()[rows.cpu().long()], torch.arange(400001).int())


@gpu
@pytest.mark.parametrize("P", [100, 5000])
def test_group_without_what_is_not_wanted(P):
    """The C call with bounds alone, and with counts beside them."""
    eidx = torch.randint(-1, 7, (P,), generator=gen(P)).int()
    dev, bounds, counts = eidx.cuda(), torch.full((8,), -77, dtype=torch.int32, device="cuda"), torch.zeros(7, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, mp.moe_group_workspace_size(P, 7)), dtype=torch.uint8, device="cuda")
    a = group_args(eidx=dev.data_ptr(), n_pairs=P, n_groups=7, bounds=bounds.data_ptr(), rows=None, pos=None, counts=counts.data_ptr(),
                   workspace=ws.data_ptr(), workspace_bytes=ws.numel())
    want = table(eidx, 7)
    for c in (counts.data_ptr(), None):
        a.counts = c
        bounds.fill_(-77)
        assert mp.lib().moe_group_rows(a, torch.cuda.current_stream().cuda_stream) == mp.MOE_OK
        assert torch.equal(bounds.cpu(), want[0]) and torch.equal(counts.cpu(), want[3])


@gpu
@pytest.mark.parametrize("P", [300, 20000])
def test_group_in_a_replayed_graph_and_on_two_streams(P):
    g, E = gen(P), 37
    eidx = torch.randint(-1, E, (P,), generator=g).int().cuda()
    ws = torch.empty(max(1, mp.moe_group_workspace_size(P, E)), dtype=torch.uint8, device="cuda")
    out = [torch.empty(n, dtype=torch.int32, device="cuda") for n in (E + 1, P, P)]
    run = lambda: mp.moe_group_rows(eidx, E, *out, workspace=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        new = torch.randint(-1, E, (P,), generator=g).int()
        eidx.copy_(new)
        for t in out:
            t.fill_(-77)
        graph.replay()
        want = table(new, E)
        n = int(want[0][-1])
        assert torch.equal(out[0].cpu(), want[0]) and torch.equal(out[1][:n].cpu(), want[1]) and torch.equal(out[2].cpu(), want[2]), i
        assert (out[1][n:] == -77).all()
    sides, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    ids = [torch.randint(-1, E, (P,), generator=g).int() for _ in range(2)]
    for side, e in zip(sides, ids):
        e = e.cuda()
        side.wait_stream(torch.cuda.current_stream())
        got.append(mp.moe_group_rows(e, E, stream=side))
    torch.cuda.synchronize()
    for (b, r, p), e in zip(got, ids):
        want = table(e, E)
        assert torch.equal(b.cpu(), want[0]) and torch.equal(p.cpu(), want[2]) and torch.equal(r[:int(b[-1])].cpu(), want[1])


# ------------------------------------------------------------------ product ---

def normal(g, dtype, *shape):
    return torch.randn(*shape, generator=g).to(dtype)


def run_product(a, b, dtype, out_dtype, bounds=None, rows=None, k=1, swiglu=False, pads=(0, 0)):
    """a [A, K], b [G, NB, K] on the host; checked, and what lies around the output too."""
    M = rows.numel() if rows is not None else a.shape[0] * k
    N = b.shape[1] // (2 if swiglu else 1)
    ad, _ = strided(a, pads[0])
    bb = torch.full((b.shape[0], b.shape[1], b.shape[2] + pads[0]), 77.0, dtype=dtype, device="cuda")
    bd = bb[..., : b.shape[2]]
    bd.copy_(b)
    buf = torch.full((M + 4, N + pads[1]), 77.0, dtype=out_dtype, device="cuda")
    out = buf[2:M + 2, :N]
    if bounds is None:
        bd = bd[0]
    mp.moe_grouped_gemm(ad, bd, out, bounds=bounds.cuda() if bounds is not None else None,
                        rows=rows.cuda() if rows is not None else None, top_k=k, swiglu=swiglu)
    want, err = ref.mx_product(a.double(), b.double(), bounds, rows, k, swiglu)
    lo, hi = (int(bounds[0]), int(bounds[-1])) if bounds is not None else (0, M)
    check_product(out[lo:hi], out_dtype, want[lo:hi], err[lo:hi])
    assert (out[:lo] == 77).all() and (out[hi:] == 77).all()
    assert (buf[:2] == 77).all() and (buf[-2:] == 77).all() and (buf[:, N:] == 77).all()


@gpu
@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
                                             (torch.float16, torch.float32)])
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (1, 64, 64), (1, 33, 2048), (2, 100, 96), (15, 31, 168), (16, 32, 256), (17, 129, 520),
                                   (33, 64, 544), (64, 65, 128), (65, 257, 1000), (130, 300, 768), (257, 255, 1024), (300, 512, 1056)])
def test_dense_product(M, N, K, dtype, out_dtype, swiglu):
    g = gen(M + N + K)
    run_product(normal(g, dtype, M, K), normal(g, dtype, 1, 2 * N if swiglu else N, K) / math.sqrt(K), dtype, out_dtype, swiglu=swiglu,
                pads=(8 * (M % 3), M % 5))


@gpu
@pytest.mark.parametrize("kind", ["one", "even", "part", "random"])
@pytest.mark.parametrize("M,N,K,G,k,gather,swiglu,dtype", [
    (8, 40, 64, 5, 2, True, True, torch.bfloat16), (40, 70, 160, 7, 4, True, False, torch.float16),
    (129, 96, 256, 3, 1, False, False, torch.bfloat16), (192, 130, 512, 20, 3, True, True, torch.float16),
    (700, 257, 296, 9, 7, False, False, torch.bfloat16), (1500, 64, 128, 64, 5, True, True, torch.bfloat16),
    (900, 300, 2048, 2, 1, True, False, torch.float16)])
def test_grouped_product(kind, M, N, K, G, k, gather, swiglu, dtype):
    g = gen(M + N + K + G)
    A = -(-M // k)
    M = A * k
    bounds = groups_of(kind, G, M, g)
    rows = torch.randperm(M, generator=g).int() if gather else None
    run_product(normal(g, dtype, A, K), normal(g, dtype, G, 2 * N if swiglu else N, K) / math.sqrt(K), dtype,
                torch.float32 if G % 2 else dtype, bounds, rows, k, swiglu, (8, 3))


@gpu
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("swiglu,out32", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("M,N,K", [(2500, 2700, 320), (3500, 3600, 128), (1200, 2500, 1000), (4100, 1030, 448), (5000, 5000, 200)])
def test_large_products(M, N, K, swiglu, out32, dtype):
    g = torch.Generator(device="cuda").manual_seed(M + K)
    a = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    b = (torch.randn(2 * N if swiglu else N, K, generator=g, device="cuda") / math.sqrt(K)).to(dtype)
    out_dtype = torch.float32 if out32 else dtype
    buf = torch.full((M, N + 3), 77.0, dtype=out_dtype, device="cuda")
    out = mp.moe_grouped_gemm(a, b, buf[:, :N], swiglu=swiglu)
    want, err = ref.mx_product(a.double(), b.double()[None], swiglu=swiglu)
    check_product(out, out_dtype, want.cpu(), err.cpu())
    assert (buf[:, N:] == 77).all()


@gpu
@pytest.mark.parametrize("M,G,k,N,K,swiglu", [(9000, 20, 3, 1500, 96, False), (6000, 40, 2, 1100, 256, True), (5000, 70, 1, 900, 160, False),
                                              (4000, 256, 8, 640, 200, True), (30000, 6, 2, 512, 64, False)])
def test_large_grouped_products(M, G, k, N, K, swiglu):
    g = gen(M + G)
    dtype = torch.bfloat16
    a, b = normal(g, dtype, M // k, K), normal(g, dtype, G, 2 * N if swiglu else N, K) / math.sqrt(K)
    M = M // k * k
    bounds, rows = groups_of("random", G, M, g), torch.randperm(M, generator=g).int()
    out = torch.full((M, N), 77.0, dtype=dtype, device="cuda")
    mp.moe_grouped_gemm(a.cuda(), b.cuda(), out, bounds=bounds.cuda(), rows=rows.cuda(), top_k=k, swiglu=swiglu)
    want, err = ref.mx_product(a.double().cuda(), b.double().cuda(), bounds, rows, k, swiglu)
    check_product(out, dtype, want.cpu(), err.cpu())


@gpu
def test_indices_outside_are_clamped_and_stay_inside():
    g = gen(5)
    a, b = normal(g, torch.bfloat16, 6, 64), normal(g, torch.bfloat16, 3, 32, 64)
    rows = torch.tensor([-5, 3, 1 << 30, 0], dtype=torch.int32)
    out = torch.full((6, 32), 77.0, device="cuda")
    mp.moe_grouped_gemm(a.cuda(), b.cuda(), out[:4], rows=rows.cuda(), bounds=torch.tensor([0, 2, 2, 4], dtype=torch.int32).cuda())
    want, err = ref.mx_product(a.double(), b.double(), torch.tensor([0, 2, 2, 4]), rows.clamp(0, 5))
    check_product(out[:4], torch.float32, want, err)
    assert (out[4:] == 77).all()


@gpu
@pytest.mark.parametrize("M,N", [(4, 32), (700, 64), (30000, 400)])
def test_bounds_that_are_not_sound_stay_inside(M, N):
    """Groups that overlap, run backwards or leave [0, M]: the rows before and behind out[5:M + 5] and the
    columns beside it keep what they held."""
    g = gen(8)
    a, b = normal(g, torch.bfloat16, M, 64).cuda(), normal(g, torch.bfloat16, 5, N, 64).cuda()
    buf = torch.full((M + 10, N + 8), 77.0, device="cuda")
    out = buf[5:M + 5, :N]
    for bad in ([0, M, 0, M, 0, M], [-7, 2, M + 9, 4, M, M], [M, M // 2, M // 3, M // 4, 1, 0], [0, 1 << 30, -(1 << 30), 1 << 30, M, 2 * M],
                [M // 2, M // 2, M + 1, 1 << 30, 1 << 30, 1 << 30], [-(1 << 31), (1 << 31) - 1, -(1 << 31), (1 << 31) - 1, 0, M]):
        mp.moe_grouped_gemm(a, b, out, bounds=torch.tensor(bad).int().cuda())
        torch.cuda.synchronize()
        assert (buf[:5] == 77).all() and (buf[M + 5:] == 77).all() and (buf[:, N:] == 77).all()


@gpu
@pytest.mark.parametrize("M,N,K,G", [(3000, 300, 512, 12), (9000, 1100, 288, 40), (60, 200, 256, 6)])
def test_grouped_product_in_a_replayed_graph_with_other_bounds(M, N, K, G):
    """What the rows are is read when the graph runs, not when it is captured."""
    g = gen(M)
    a, b = normal(g, torch.float16, M, K).cuda(), (normal(g, torch.float16, G, 2 * N, K) / 16).cuda()
    bounds, rows = groups_of("even", G, M, g).cuda(), torch.arange(M).int().cuda()
    out = torch.full((M, N), 77.0, dtype=torch.float16, device="cuda")
    run = lambda o: mp.moe_grouped_gemm(a, b, o, bounds=bounds, rows=rows, swiglu=True)  # noqa: E731
    run(torch.empty_like(out))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for kind in ("random", "one", "part", "even"):
        bounds.copy_(groups_of(kind, G, M, g))
        rows.copy_(torch.randperm(M, generator=g).int())
        out.fill_(77.0)
        graph.replay()
        want = torch.full_like(out, 77.0)
        run(want)
        torch.cuda.synchronize()
        assert torch.equal(out, want), kind


@gpu
@pytest.mark.parametrize("M,N,K", [(40, 70, 200), (700, 900, 136), (300, 600, 128), (4200, 4200, 72)])
def test_infinities_and_nan_reach_their_rows_and_columns_only(M, N, K):
    """Also in the last values of K, which lie next to what a tile reads past its end."""
    g = gen(6)
    a, b = normal(g, torch.bfloat16, M, K), normal(g, torch.bfloat16, 1, N, K)
    a[3, 2], a[M - 1, K - 1] = math.nan, math.inf
    b[0, N // 2, K - 1], b[0, 1, 0] = math.nan, -math.inf
    out = mp.moe_grouped_gemm(a.cuda(), b[0].cuda(), dtype=torch.float32).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[3] = bad[M - 1] = True
    bad[:, N // 2] = bad[:, 1] = True
    assert not torch.isfinite(out[bad]).any() and torch.isfinite(out[~bad]).all()
    fine = torch.isfinite(a).all(1)[:, None] & torch.isfinite(b[0]).all(1)[None]
    want, err = ref.mx_product(a.double().nan_to_num(0, 0, 0), b.double().nan_to_num(0, 0, 0))
    got = out.double()
    assert ((got - want).abs() <= err + 2.0 ** -24 * (want.abs() + err))[fine].all()


@gpu
@pytest.mark.parametrize("far,M", [("a", 5), ("a just below", 130), ("a", 130), ("b", 3), ("b", 70), ("out", 70), ("stride", 200), ("b stride", 200)])
def test_offsets_past_32_bits(far, M):
    """A (reached by a row table), B or their rows' strides that span more than 2^32 bytes, or just fewer, and an
    output that does: all zero but for the rows that count."""
    g = gen(M)
    K = 64 if far in ("out", "stride", "b stride") else 1 << 16
    A = {"a": 32800, "a just below": 32767}.get(far, M)
    N = 33000 if far == "b" else 300 if far == "b stride" else 40
    step = {"stride": 1 << 24, "b stride": 1 << 24}.get(far, K)
    a = torch.zeros((A - 1) * (step if far == "stride" else K) + K, dtype=torch.bfloat16, device="cuda").as_strided((A, K), (step if far == "stride" else K, 1))
    b = torch.zeros((N - 1) * (step if far == "b stride" else K) + K, dtype=torch.bfloat16, device="cuda").as_strided((N, K), (step if far == "b stride" else K, 1))
    ar = sorted({0, A // 2, A - 2, A - 1}) if A > M else list(range(M))
    br = [0, N // 2, N - 1]
    for t, rows in ((a, ar), (b, br)):
        v = normal(g, torch.bfloat16, len(rows), K).cuda()
        for i, r in enumerate(rows):
            t[r] = v[i]
    rows = torch.tensor(ar)[torch.randint(0, len(ar), (M,), generator=g)].int().cuda() if A > M else None
    stride = 1 << 26 if far == "out" else N
    buf = torch.empty((M - 1) * stride + N, device="cuda")
    out = buf.as_strided((M, N), (stride, 1))
    mp.moe_grouped_gemm(a, b, out, rows=rows)
    near = torch.searchsorted(torch.tensor(ar), rows.cpu().long()).int() if rows is not None else None
    want, err = ref.mx_product(a[ar].double().cpu(), b[br].double().cpu()[None], rows=near)
    check_product(out[:, br], torch.float32, want, err)
    zero = torch.ones(N, dtype=torch.bool)
    zero[br] = False
    assert (out[:, zero.cuda()] == 0).all()


@gpu
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_empty_groups(swiglu):
    """More groups than are scanned at a time, nearly all of them without rows; one matrix for all of them."""
    g = gen(11)
    G, M, N, K = 65535, 900, 150, 40
    a, one = normal(g, torch.bfloat16, M, K), normal(g, torch.bfloat16, 2 * N, K)
    b = one.cuda()[None].expand(G, -1, -1)                # the groups' stride is 0
    held = sorted(torch.randperm(G, generator=g)[:12].tolist())
    cuts = [0] + sorted(torch.randint(0, M + 1, (11,), generator=g).tolist()) + [M]
    bounds = torch.zeros(G + 1, dtype=torch.int32)
    for i, e in enumerate(held):
        bounds[e + 1:] = cuts[i + 1]
    out = torch.full((M, N if swiglu else 2 * N), 77.0, device="cuda")
    mp.moe_grouped_gemm(a.cuda(), b, out, bounds=bounds.cuda(), swiglu=swiglu)
    want, err = ref.mx_product(a.double(), one.double()[None], swiglu=swiglu)
    check_product(out, torch.float32, want, err)


@gpu
def test_products_on_two_streams_at_once():
    g = gen(6)
    sets = []
    for M, N, K in ((700, 900, 1024), (2500, 4200, 512)):
        a, b = normal(g, torch.bfloat16, M, K).cuda(), normal(g, torch.bfloat16, N, K).cuda()
        sets.append((a, b, mp.moe_grouped_gemm(a, b)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(4):
        for (a, b, want), s in zip(sets, streams):
            o = torch.full_like(want, 77.0)
            s.wait_stream(torch.cuda.current_stream())
            mp.moe_grouped_gemm(a, b, o, stream=s)
            outs.append((o, want))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in outs)


# ------------------------------------------------------------------ combine ---

def combine_reference(d, w, pos, base):
    """(y, bound): k + 1 roundings of 2^-24 of the sum of magnitudes."""
    d, w = d.double(), w.double()
    live = (pos >= 0) & (pos < d.shape[0])
    y = base.double().clone() if base is not None else torch.zeros(pos.shape[0], d.shape[1], dtype=torch.float64)
    mag = y.abs()
    for j in range(pos.shape[1]):
        at = live[:, j].nonzero().flatten()
        row = d[pos[at, j].long()] * w[at, j, None]
        y[at] += row
        mag[at] += row.abs()
    return y, (pos.shape[1] + 1) * 2.0 ** -24 * mag


@gpu
@pytest.mark.parametrize("d_type", ALL)
@pytest.mark.parametrize("y_type", ALL)
@pytest.mark.parametrize("T,N,k,R,pad,base_type", [
    (1, 8, 1, 1, 0, None), (1, 2048, 8, 8, 0, torch.float32), (3, 33, 2, 6, 1, torch.bfloat16), (70, 512, 9, 500, 8, torch.float16),
    (257, 129, 3, 700, 0, torch.float32), (65, 1000, 17, 64, 24, torch.bfloat16), (1000, 64, 4, 4000, 0, None), (5, 5000, 8, 40, 4, torch.float32)])
def test_combine(T, N, k, R, pad, base_type, d_type, y_type):
    g = gen(T + N)
    d, w = torch.randn(R, N, generator=g).to(d_type), torch.randn(T, k, generator=g)
    pos = torch.randint(-2, R + 2, (T, k), generator=g).int()
    pos[T // 2] = -1                                      # a token with no expert
    base = torch.randn(T, N, generator=g).to(base_type) if base_type else None
    dd, _ = strided(d, pad)
    y, buf = strided(torch.zeros(T, N, dtype=y_type), pad)
    bd = strided(base, pad)[0] if base_type else None
    want, err = combine_reference(d, w, pos, base)
    mp.moe_combine_rows(dd, w.cuda(), pos.cuda(), y, base=bd)
    got = y.double().cpu()
    tol = err + ref.half_step(y_type) * (want.abs() + err) + ref.least_step(y_type)
    assert ((got - want).abs() <= tol).all()
    assert (buf[:, N:] == 77).all()
    if pad == 0:
        assert torch.equal(mp.moe_combine_rows(dd, w.cuda(), pos.cuda(), base=bd, dtype=y_type), y)
    if base_type == y_type:                               # in place: the same bits
        mp.moe_combine_rows(dd, w.cuda(), pos.cuda(), bd, base=bd)
        assert torch.equal(bd, y)


@gpu
def test_combine_leaves_masked_rows_out():
    """What a masked slot's weight is, and what rows that no slot names hold, does not matter."""
    d = torch.full((4, 40), math.nan, device="cuda")
    d[1] = 2.0
    w = torch.tensor([[0.5, math.nan], [math.inf, 3.0], [1.0, -math.inf]], device="cuda")
    pos = torch.tensor([[1, -1], [-1, 1], [7, -(1 << 31)]], dtype=torch.int32, device="cuda")
    y = mp.moe_combine_rows(d, w, pos)
    assert (y == torch.tensor([1.0, 6.0, 0.0], device="cuda")[:, None]).all()
    assert (mp.moe_combine_rows(d[:0], w, pos) == 0).all()


@gpu
def test_combine_past_32_bits():
    R, N = 70000, 32768                                   # 2.3 G elements of d
    d = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    d[R - 1] = 3.0
    d[65537] = 5.0
    pos = torch.tensor([[R - 1, 65537]], dtype=torch.int32, device="cuda")
    assert (mp.moe_combine_rows(d, torch.tensor([[1.0, 2.0]], device="cuda"), pos) == 13).all()


# ----------------------------------------------------------------- together ---

@gpu
@pytest.mark.parametrize("T,E,k", [(3, 8, 2), (150, 10, 3), (900, 16, 4)])
def test_a_layer_of_16_bit_experts_beside_a_shared_one(T, E, k):
    """Routing by a sigmoid router (not the prompt layer's), row table, gate/up with SwiGLU, down, and the
    combine onto a shared expert's output; a slot of the batch and one expert left out."""
    d, f = 256, 192
    g = gen(T)
    bf = torch.bfloat16
    x = torch.randn(T, d, generator=g).to(bf).cuda()
    scores = torch.sigmoid(torch.randn(T, E, generator=g))
    scores[:, E - 1] = -1.0
    top = scores.topk(k, -1)
    eidx, w = top.indices.int(), top.values / top.values.sum(-1, keepdim=True)
    eidx[T // 2] = -1
    eidx, w = eidx.cuda(), w.cuda()
    gu, dn = [(torch.randn(E + 1, *s, generator=g) / 16).to(bf).cuda() for s in ((2 * f, d), (d, f))]    # the last: shared
    bounds, rows, pos = mp.moe_group_rows(eidx, E)
    h = mp.moe_grouped_gemm(x, gu[:E], bounds=bounds, rows=rows, top_k=k, swiglu=True)
    dm = mp.moe_grouped_gemm(h, dn[:E], bounds=bounds, dtype=torch.float32)
    shared = mp.moe_grouped_gemm(mp.moe_grouped_gemm(x, gu[E], swiglu=True), dn[E], dtype=torch.float32)
    y = mp.moe_combine_rows(dm, w, pos, base=shared)
    # each stage from the values of the one before
    n = int(bounds[-1])
    want, err = ref.mx_product(x.double().cpu(), gu[:E].double().cpu(), bounds, rows[:n], k, True)
    check_product(h[:n], bf, want, err)
    want, err = ref.mx_product(h[:n].double().cpu(), dn[:E].double().cpu(), bounds)
    check_product(dm[:n], torch.float32, want, err)
    want, err = combine_reference(dm.cpu(), w.cpu(), pos.cpu(), shared.cpu())
    assert ((y.double().cpu() - want).abs() <= err + 2.0 ** -24 * (want.abs() + err)).all()
    assert torch.equal(y[T // 2], shared[T // 2])
    # by the dense formula: h is rounded to bf16 (2^-9 of its size at the root mean square) before the down product
    x, wgu, wdn = x.double().cpu(), gu.double().cpu(), dn.double().cpu()

    def expert(e, v):
        z = wgu[e] @ v
        return wdn[e] @ (z[:f] * torch.sigmoid(z[:f]) * z[f:])

    full = torch.stack([expert(E, v) for v in x])
    for t in range(T):
        for j, e in enumerate(eidx[t].tolist()):
            if e >= 0:
                full[t] += w[t, j].double().cpu() * expert(e, x[t])
    assert float((y.double().cpu() - full).norm() / full.norm()) < 2.0 ** -8


@gpu
def test_mxfp4_product_over_a_table_of_any_routing():
    from test_mxfp4 import random_mx
    g = gen(2)
    T, E, k, N, K = 90, 12, 3, 70, 128
    eidx = torch.randint(-1, E, (T, k), generator=g).int()
    a, b = random_mx(g, T, K, hi=120), random_mx(g, E, N, K, hi=120)
    bounds, rows, _ = mp.moe_group_rows(eidx.cuda(), E)
    out = mp.moe_mxfp4_gemm(*[t.cuda() for t in (*a, *b)], bounds=bounds, rows=rows, top_k=k)
    n = int(bounds[-1])
    want, err = ref.mx_product(ref.mx_values(*a), ref.mx_values(*b), bounds, rows[:n], k)
    check_product(out[:n], torch.float32, want, err)


@gpu
def test_the_table_is_the_one_that_the_prompt_layer_exports():
    d, f, E, k, T = 64, 64, 12, 4, 333
    g = gen(4)
    R = T * k
    ex = {n: torch.empty(s, dtype=torch.int32, device="cuda") for n, s in (("rows", R), ("pos", R), ("eidx", R), ("bounds", E + 1), ("counts", E))}
    h = mp.moe_prefill_create(d, f, E, k, T)
    blob = torch.zeros(mp.moe_prefill_layer_bytes(d, f, E), dtype=torch.uint8, device="cuda")
    y = torch.empty(T, d, device="cuda")
    mp.moe_prefill_run_layer(h, torch.randn(T, d, generator=g).cuda(), torch.randn(T, E, generator=g).cuda(), y, weights=blob, exports=ex)
    counts = torch.empty(E, dtype=torch.int32, device="cuda")
    bounds, rows, pos = mp.moe_group_rows(ex["eidx"], E, counts=counts)
    torch.cuda.synchronize()
    h.close()
    for name, t in (("bounds", bounds), ("rows", rows), ("pos", pos), ("counts", counts)):
        assert torch.equal(ex[name], t), name


@gpu
def test_binding_refusals_on_the_device():
    z = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for bad in (lambda: mp.moe_grouped_gemm(z, z[:, :32]), lambda: mp.moe_grouped_gemm(z, z[None].expand(2, -1, -1)),
                lambda: mp.moe_grouped_gemm(z, z[:3], swiglu=True), lambda: mp.moe_grouped_gemm(z, z, top_k=0),
                lambda: mp.moe_grouped_gemm(z, z, torch.zeros(4, 5, dtype=torch.bfloat16, device="cuda")),
                lambda: mp.moe_grouped_gemm(z, z, bounds=i.view(-1)[:3]), lambda: mp.moe_grouped_gemm(z, z.t()),
                lambda: mp.moe_grouped_gemm(z, z.as_strided((4, 64), (32, 1))),
                lambda: mp.moe_group_rows(i, 4, bounds=i[0]), lambda: mp.moe_group_rows(i, 4, rows=i[0]),
                lambda: mp.moe_combine_rows(z, torch.zeros(4, 3, device="cuda"), i)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: mp.moe_grouped_gemm(z.float(), z.float()), lambda: mp.moe_grouped_gemm(z, z.half()),
                lambda: mp.moe_grouped_gemm(z, z, dtype=torch.float16), lambda: mp.moe_grouped_gemm(z, z.cpu()),
                lambda: mp.moe_grouped_gemm(z, z, rows=torch.zeros(4, dtype=torch.int64, device="cuda")),
                lambda: mp.moe_group_rows(i.long(), 4), lambda: mp.moe_group_rows(i.t(), 4),
                lambda: mp.moe_combine_rows(z, torch.zeros(4, 2, device="cuda"), i.long()),
                lambda: mp.moe_combine_rows(z.double(), torch.zeros(4, 2, device="cuda"), i)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(mp.MoePrefillError):
        mp.moe_grouped_gemm(z[:, :60], z[:, :60])         # K no multiple of 8
    with pytest.raises(mp.MoePrefillError):
        mp.moe_grouped_gemm(z.view(-1)[4:68].view(1, 64), z)    # rows not 16-byte aligned
    assert mp.moe_grouped_gemm(z[:0], z).shape == (0, 4)
    assert mp.moe_combine_rows(z, torch.zeros(0, 2, device="cuda"), i[:0]).shape == (0, 64)
