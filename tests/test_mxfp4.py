"""MXFP4: quantise, dequantise and the product (dense, grouped, gathered, SwiGLU) against
plain 64-bit forms, at the sizes and values where they can go wrong, and their refusals."""
import ctypes
import math

import pytest
import torch

import moe_prefill_ffn_amd as mp
import mx_reference as ref

gpu = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def gen(seed):
    return torch.Generator().manual_seed(seed)


def strided(t, pad, dev="cuda:0"):
    """t on the device, its rows in a wider buffer of sentinels; (view, buffer)."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), 77.0).to(t.dtype).to(dev)
    buf[:, : t.shape[1]] = t.to(dev)
    return buf[:, : t.shape[1]], buf


# ----------------------------------------------------------- refusals (CPU) ---

def matrix(**kw):
    m = mp.moe_mxfp4_matrix_t()
    m.struct_size = ctypes.sizeof(m)
    m.dtype, m.K, m.M, m.stride = mp.MOE_F32, 64, 4, 64
    m.values, m.codes, m.scales = 4096, 8192, 16384     # never read: every case below is refused first
    for k, v in kw.items():
        setattr(m, k, v)
    return m


@pytest.mark.parametrize("bad", [
    dict(struct_size=4), dict(dtype=3), dict(dtype=-1), dict(K=0), dict(K=33), dict(K=-32), dict(M=-1),
    dict(M=1 << 31), dict(M=1 << 29), dict(K=1 << 20, M=1 << 15, stride=1 << 20), dict(values=None), dict(codes=None), dict(scales=None), dict(stride=63), dict(stride=-64),
    dict(stride=1 << 41), dict(values=4100), dict(codes=8200), dict(stride=66), dict(stride=68, dtype=mp.MOE_BF16)])
def test_matrix_refusals(bad):
    for fn in (mp.lib().moe_mxfp4_quantize, mp.lib().moe_mxfp4_dequantize):
        assert fn(matrix(**bad), None) == mp.MOE_EINVAL
        assert mp.moe_prefill_last_error()


def test_matrix_of_no_rows_is_a_no_op_without_pointers():
    assert mp.lib().moe_mxfp4_quantize(matrix(M=0, values=None, codes=None, scales=None), None) == mp.MOE_OK
    assert mp.lib().moe_mxfp4_dequantize(matrix(M=0, values=None, codes=None, scales=None), None) == mp.MOE_OK


def gemm_args(**kw):
    a = mp.moe_mxfp4_gemm_args_t()
    a.struct_size = ctypes.sizeof(a)
    a.a_codes, a.a_scales, a.b_codes, a.b_scales, a.out = 4096, 8192, 16384, 32768, 65536
    a.a_rows, a.n_groups, a.top_k, a.M, a.N, a.K, a.out_stride = 4, 1, 1, 4, 8, 64, 8
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("bad", [
    dict(struct_size=0), dict(dtype=7), dict(swiglu=2), dict(K=0), dict(K=48), dict(K=(1 << 20) + 32), dict(N=0), dict(N=1 << 21), dict(M=-1),
    dict(M=1 << 31), dict(M=(1 << 27) + 1, a_rows=1 << 28), dict(M=1 << 24, a_rows=1 << 24, N=1 << 20, out_stride=1 << 20),
    dict(a_rows=1 << 31), dict(n_groups=0), dict(n_groups=2), dict(n_groups=65536, bounds=128), dict(top_k=0),
    dict(a_codes=None), dict(a_scales=None), dict(b_codes=None), dict(b_scales=None), dict(out=None),
    dict(a_rows=0), dict(a_rows=3), dict(a_rows=1, top_k=3), dict(a_rows=0, rows=128), dict(out_stride=7),
    dict(a_codes=4104), dict(b_codes=16400 - 8), dict(out=65538), dict(out=65537, dtype=mp.MOE_BF16),
    dict(bounds=130), dict(rows=129)])
def test_gemm_refusals(bad):
    assert mp.lib().moe_mxfp4_gemm(gemm_args(**bad), None) == mp.MOE_EINVAL
    assert mp.moe_prefill_last_error()


def test_gemm_of_no_rows_is_a_no_op_without_pointers():
    a = gemm_args(M=0, a_codes=None, a_scales=None, b_codes=None, b_scales=None, out=None, a_rows=0)
    assert mp.lib().moe_mxfp4_gemm(a, None) == mp.MOE_OK


def test_binding_refuses_host_tensors():
    with pytest.raises(TypeError):
        mp.moe_mxfp4_quantize(torch.zeros(2, 64))
    with pytest.raises(TypeError):
        mp.moe_mxfp4_dequantize(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 2, dtype=torch.uint8))
    with pytest.raises(TypeError):
        z = torch.zeros(2, 32, dtype=torch.uint8)
        mp.moe_mxfp4_gemm(z, z[:, :2], z, z[:, :2])


# ------------------------------------------------------- quantise, and back ---

def special_rows(dtype):
    """Rows of 64: ties, neighbours of the borders, zeros, the type's range, infinities, NaN."""
    fin = torch.finfo(dtype)
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375])
    tie = torch.cat([ties, -ties, torch.zeros(11), torch.tensor([4.0])])
    rows = [torch.cat([tie, tie * 2.0 ** -6]),
            torch.zeros(64), -torch.zeros(64),
            torch.cat([torch.full((32,), fin.max), torch.full((32,), fin.tiny)]),
            torch.cat([torch.full((32,), -fin.max), torch.full((32,), fin.smallest_normal * 2.0 ** -4)]),
            torch.arange(64) * 1.0, torch.where(torch.arange(64) == 5, math.inf, 1.0),
            torch.where(torch.arange(64) == 40, math.nan, 1.0), torch.where(torch.arange(64) == 63, -math.inf, 0.0),
            torch.cat([torch.full((32,), 1.0), torch.full((32,), fin.smallest_normal)])]
    return torch.stack([r.double() for r in rows]).to(dtype)


def assert_same(got, want):
    """Equal values, NaN in the same places (blocks that held an infinity or a NaN)."""
    got = got.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~torch.isnan(got)], want[~torch.isnan(want)])


def check_quantised(x_dev, codes, scales, dtype):
    rc, rs = ref.mx_quantize(x_dev)
    assert torch.equal(scales.cpu(), rs)
    assert torch.equal(codes.cpu(), rc)
    assert_same(mp.moe_mxfp4_dequantize(codes, scales, dtype=dtype), ref.mx_values(rc, rs).to(dtype))


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantise_special_values(dtype):
    x = special_rows(dtype).cuda()
    codes, scales = mp.moe_mxfp4_quantize(x)
    check_quantised(x, codes, scales, dtype)


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,K,pad", [(1, 32, 0), (1, 2048, 8), (3, 96, 16), (5, 1504, 40), (257, 32, 8), (64, 4096, 0), (1021, 160, 0)])
def test_quantise_shapes_and_strides(dtype, M, K, pad):
    x = (torch.randn(M, K, generator=gen(M + K)) * torch.exp(3 * torch.randn(M, 1, generator=gen(7)))).to(dtype)
    xd, buf = strided(x, pad)
    codes, scales = mp.moe_mxfp4_quantize(xd)
    check_quantised(xd, codes, scales, dtype)
    out, obuf = strided(torch.zeros(M, K, dtype=dtype), pad)
    mp.moe_mxfp4_dequantize(codes, scales, out)
    assert_same(out, ref.mx_values(codes, scales).to(dtype))
    assert (obuf[:, K:] == 77).all()                      # nothing between the rows


@gpu
def test_dequantise_every_code_and_scale():
    codes = torch.arange(256).repeat_interleave(16).reshape(256, 16).to(torch.uint8)
    codes = torch.stack([(codes + 17 * i) for i in range(16)], 0).reshape(-1, 16).to(torch.uint8)
    scales = torch.arange(256).repeat(16).reshape(-1, 1).to(torch.uint8)
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        # fp64 -> fp32 is exact, or infinity past 2^128
        assert_same(mp.moe_mxfp4_dequantize(codes.cuda(), scales.cuda(), dtype=dtype),
                    ref.mx_values(codes, scales).float().to(dtype))


# ------------------------------------------------------------------ product ---

def random_mx(g, *shape, lo=110, hi=130):
    K = shape[-1]
    return (torch.randint(0, 256, (*shape[:-1], K // 2), generator=g).to(torch.uint8),
            torch.randint(lo, hi, (*shape[:-1], K // 32), generator=g).to(torch.uint8))


def check_product(out, dtype, want, err):
    got = out.double().cpu()
    tol = err + ref.half_step(dtype) * (want.abs() + err) + ref.least_step(dtype)
    assert torch.isfinite(want).all()
    bad = (got - want).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float((got - want).abs().max()))
    # what the sums' roundings come to together, and the least step of every element (an fp16
    # output of 1e-8 is 0)
    assert float((got - want).norm()) <= (2e-6 + 1.2 * ref.half_step(dtype)) * float(want.norm()) + ref.least_step(dtype) * got.numel() ** 0.5


@gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("M,N,K", [(1, 1, 32), (1, 64, 64), (1, 33, 2048), (2, 100, 96), (15, 31, 160), (16, 32, 256), (17, 129, 512),
                                   (33, 64, 544), (64, 65, 128), (65, 257, 992), (130, 300, 768), (257, 255, 1024), (300, 512, 1056)])
def test_dense_product(M, N, K, dtype, swiglu):
    g = gen(M * 7 + N * 3 + K)
    NB = 2 * N if swiglu else N
    hi = 122 if dtype == torch.float16 or swiglu else 130
    ac, asc = random_mx(g, M, K, hi=hi)
    bc, bsc = random_mx(g, NB, K, hi=hi)
    out, buf = strided(torch.zeros(M, N, dtype=dtype), 3)
    r = mp.moe_mxfp4_gemm(ac.cuda(), asc.cuda(), bc.cuda(), bsc.cuda(), out, swiglu=swiglu)
    assert r is out
    want, err = ref.mx_product(ref.mx_values(ac, asc), ref.mx_values(bc, bsc)[None], swiglu=swiglu)
    check_product(out, dtype, want, err)
    assert (buf[:, N:] == 77).all()


@gpu
@pytest.mark.parametrize("K", [128, 384, 480, 512, 1536])  # scale rows 16-byte aligned, 4-byte aligned, and not
@pytest.mark.parametrize("swiglu,dtype", [(False, torch.bfloat16), (True, torch.float32), (False, torch.float32)])
@pytest.mark.parametrize("M,N", [(3500, 3600), (1200, 2500), (4100, 1030), (5000, 7000)])
def test_large_products_take_the_wider_tiles(M, N, K, swiglu, dtype):
    """Row and column counts of no tile's multiple, at which each of the wider tiles is chosen."""
    g = gen(M + N + K)
    N = N // 2 if swiglu else N
    ac, asc = random_mx(g, M, K, hi=122)
    bc, bsc = random_mx(g, 2 * N if swiglu else N, K, hi=122)
    out = torch.full((M + 2, N), 77.0, dtype=dtype, device="cuda")
    mp.moe_mxfp4_gemm(ac.cuda(), asc.cuda(), bc.cuda(), bsc.cuda(), out[:M], swiglu=swiglu)
    want, err = ref.mx_product(ref.mx_values(ac, asc).cuda(), ref.mx_values(bc, bsc)[None].cuda(), swiglu=swiglu)
    check_product(out[:M], dtype, want.cpu(), err.cpu())
    assert (out[M:] == 77).all()


@gpu
@pytest.mark.parametrize("K", [2048, 2080, 2176])         # scale rows 16-byte aligned, not at all, 4-byte aligned
@pytest.mark.parametrize("M,N,swiglu,dtype", [(5000, 6100, False, torch.float32), (5001, 3050, True, torch.bfloat16)])
def test_products_of_the_widest_tiles(M, N, K, swiglu, dtype):
    g = gen(M + K)
    a = [t.cuda() for t in random_mx(g, M, K, hi=118)]
    b = [t.cuda() for t in random_mx(g, 2 * N if swiglu else N, K, hi=118)]
    out = torch.full((M + 2, N), 77.0, dtype=dtype, device="cuda")
    mp.moe_mxfp4_gemm(*a, *b, out[:M], swiglu=swiglu)
    want, err = ref.mx_product(ref.mx_values(*a).cuda(), ref.mx_values(*b)[None].cuda(), swiglu=swiglu)
    check_product(out[:M], dtype, want.cpu(), err.cpu())
    assert (out[M:] == 77).all()


@gpu
@pytest.mark.parametrize("M,G,k,N,K,swiglu", [(9000, 20, 3, 1500, 96, False), (6000, 40, 2, 1100, 256, True), (5000, 70, 1, 900, 160, False),
                                              (4001, 4, 1, 7001, 2048, False)])
def test_large_grouped_products(M, G, k, N, K, swiglu):
    g = gen(M + G)
    ac, asc = random_mx(g, M // k, K, hi=122)
    M = M // k * k
    bc, bsc = random_mx(g, G, 2 * N if swiglu else N, K, hi=122)
    bounds = groups_of("random", G, M, g)
    rows = torch.randperm(M, generator=g).int()
    out = torch.full((M, N), 77.0, device="cuda")
    mp.moe_mxfp4_gemm(ac.cuda(), asc.cuda(), bc.cuda(), bsc.cuda(), out, bounds=bounds.cuda(), rows=rows.cuda(), top_k=k, swiglu=swiglu)
    want, err = ref.mx_product(ref.mx_values(ac, asc).cuda(), ref.mx_values(bc, bsc).cuda(), bounds, rows, k, swiglu)
    check_product(out, torch.float32, want.cpu(), err.cpu())


def groups_of(kind, G, M, g):
    """Ascending bounds [G + 1] of M rows: empty groups at both ends and inside, one that holds all, ..."""
    if kind == "one":
        cuts = [0] * (G // 2 + 1) + [M] * (G - G // 2)
    elif kind == "even":
        cuts = [M * i // G for i in range(G + 1)]
    elif kind == "part":                                  # rows before the first and behind the last group
        cuts = [min(M, 3 + (M - 6) * i // G) for i in range(G + 1)]
    else:
        cuts = [0] + sorted(torch.randint(0, M + 1, (G - 1,), generator=g).tolist()) + [M]
    return torch.tensor(cuts, dtype=torch.int32)


@gpu
@pytest.mark.parametrize("kind", ["one", "even", "part", "random"])
@pytest.mark.parametrize("M,N,K,G,k,gather,swiglu,dtype", [
    (8, 40, 64, 5, 2, True, True, torch.float32), (40, 70, 160, 7, 4, True, False, torch.bfloat16),
    (129, 96, 256, 3, 1, False, False, torch.float16), (192, 130, 512, 20, 3, True, True, torch.bfloat16),
    (700, 257, 288, 9, 7, False, False, torch.float32), (1500, 64, 128, 64, 5, True, True, torch.float32),
    (900, 300, 2048, 2, 1, True, False, torch.bfloat16)])
def test_grouped_product(kind, M, N, K, G, k, gather, swiglu, dtype):
    g = gen(M + N + K + G)
    A = -(-M // k)
    M = A * k
    ac, asc = random_mx(g, A, K, hi=120)
    bc, bsc = random_mx(g, G, 2 * N if swiglu else N, K, hi=120)
    bounds = groups_of(kind, G, M, g)
    rows = torch.randperm(M, generator=g).int() if gather else None
    out = torch.full((M, N), 77.0, dtype=dtype, device="cuda")
    mp.moe_mxfp4_gemm(ac.cuda(), asc.cuda(), bc.cuda(), bsc.cuda(), out, bounds=bounds.cuda(),
                      rows=rows.cuda() if gather else None, top_k=k, swiglu=swiglu)
    want, err = ref.mx_product(ref.mx_values(ac, asc), ref.mx_values(bc, bsc), bounds, rows, k, swiglu)
    lo, hi = int(bounds[0]), int(bounds[-1])
    check_product(out[lo:hi], dtype, want[lo:hi], err[lo:hi])
    assert (out[:lo] == 77).all() and (out[hi:] == 77).all()


@gpu
def test_indices_outside_are_clamped_and_stay_inside():
    g = gen(5)
    ac, asc = random_mx(g, 6, 64)
    bc, bsc = random_mx(g, 3, 32, 64)
    rows = torch.tensor([-5, 3, 1 << 30, 0], dtype=torch.int32)
    out = torch.full((6, 32), 77.0, device="cuda")
    mp.moe_mxfp4_gemm(ac.cuda(), asc.cuda(), bc.cuda(), bsc.cuda(), out[:4], rows=rows.cuda(),
                      bounds=torch.tensor([0, 2, 2, 4], dtype=torch.int32).cuda())
    want, err = ref.mx_product(ref.mx_values(ac, asc), ref.mx_values(bc, bsc), torch.tensor([0, 2, 2, 4]), rows.clamp(0, 5))
    check_product(out[:4], torch.float32, want, err)
    assert (out[4:] == 77).all()
    # bounds that do not ascend, or leave [0, M]: nothing outside out[:4] is written
    for bad in ([0, 900, 2, 4], [-7, 2, 3, 4], [4, 3, 2, 0], [0, 1 << 30, -(1 << 30), 1 << 30]):
        mp.moe_mxfp4_gemm(ac.cuda(), asc.cuda(), bc.cuda(), bsc.cuda(), out[:4], rows=rows.cuda(),
                          bounds=torch.tensor(bad, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert (out[4:] == 77).all()


@gpu
@pytest.mark.parametrize("M,N", [(700, 64), (30000, 400)])
def test_bounds_that_are_not_sound_stay_inside(M, N):
    """Groups that overlap, run backwards or leave [0, M], in the tiled kernels: the rows before and behind
    out[5:M + 5] and the columns beside it keep what they held."""
    g = gen(8)
    a, b = [t.cuda() for t in random_mx(g, M, 64)], [t.cuda() for t in random_mx(g, 5, N, 64)]
    buf = torch.full((M + 10, N + 8), 77.0, device="cuda")
    out = buf[5:M + 5, :N]
    for bad in ([0, M, 0, M, 0, M], [-7, 2, M + 9, 4, M, M], [M, 300, 200, 100, 50, 0], [0, 1 << 30, -(1 << 30), 1 << 30, M, 2 * M],
                [M // 2, M // 2, M + 1, 1 << 30, 1 << 30, 1 << 30], [-(1 << 31), (1 << 31) - 1, -(1 << 31), (1 << 31) - 1, 0, M]):
        mp.moe_mxfp4_gemm(*a, *b, out, bounds=torch.tensor(bad).int().cuda())
        torch.cuda.synchronize()
        assert (buf[:5] == 77).all() and (buf[M + 5:] == 77).all() and (buf[:, N:] == 77).all()


@gpu
@pytest.mark.parametrize("M,N,K,G", [(3000, 300, 512, 12), (9000, 1100, 288, 40), (60, 200, 256, 6)])
def test_grouped_product_in_a_replayed_graph_with_other_bounds(M, N, K, G):
    """What the rows are is read when the graph runs, not when it is captured."""
    g = gen(M)
    a, b = [t.cuda() for t in random_mx(g, M, K, hi=120)], [t.cuda() for t in random_mx(g, G, 2 * N, K, hi=120)]
    bounds, rows = groups_of("even", G, M, g).cuda(), torch.arange(M).int().cuda()
    out = torch.full((M, N), 77.0, dtype=torch.bfloat16, device="cuda")
    run = lambda o: mp.moe_mxfp4_gemm(*a, *b, o, bounds=bounds, rows=rows, swiglu=True)  # noqa: E731
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
def test_nan_blocks_reach_their_rows_and_columns_only():
    g = gen(6)
    ac, asc = random_mx(g, 40, 128)
    bc, bsc = random_mx(g, 70, 128)
    asc[3, 2] = 255
    bsc[65, 0] = 255
    out = mp.moe_mxfp4_gemm(ac.cuda(), asc.cuda(), bc.cuda(), bsc.cuda()).cpu()
    bad = torch.isnan(out)
    want = torch.zeros(40, 70, dtype=torch.bool)
    want[3], want[:, 65] = True, True
    assert torch.equal(bad, want)


@gpu
def test_scales_at_any_byte_address():
    g = gen(8)
    ac, asc = random_mx(g, 5, 256)
    bc, bsc = random_mx(g, 9, 256)
    raw = torch.zeros(3 + asc.numel() + 1 + bsc.numel(), dtype=torch.uint8, device="cuda")
    a_s = raw[3:3 + asc.numel()].view(asc.shape)
    b_s = raw[3 + asc.numel() + 1:].view(bsc.shape)
    a_s.copy_(asc)
    b_s.copy_(bsc)
    out = mp.moe_mxfp4_gemm(ac.cuda(), a_s, bc.cuda(), b_s)
    want, err = ref.mx_product(ref.mx_values(ac, asc), ref.mx_values(bc, bsc)[None])
    check_product(out, torch.float32, want, err)


@gpu
def test_no_rows_and_no_groups_with_rows():
    g = gen(9)
    bc, bsc = random_mx(g, 4, 32, 64)
    e = torch.empty(0, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda")
    out = mp.moe_mxfp4_gemm(*e, bc.cuda(), bsc.cuda(), bounds=torch.zeros(5, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 32)
    assert mp.moe_mxfp4_quantize(torch.empty(0, 64, device="cuda"))[0].shape == (0, 32)
    a = [t.cuda() for t in random_mx(g, 5, 64)]
    out = torch.full((5, 32), 77.0, device="cuda")
    mp.moe_mxfp4_gemm(*a, bc.cuda(), bsc.cuda(), out, bounds=torch.zeros(5, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert (out == 77).all()


@gpu
def test_quantise_and_product_in_a_replayed_graph_and_on_another_stream():
    g = gen(10)
    x = torch.randn(50, 512, generator=g).cuda()
    bc, bsc = [t.cuda() for t in random_mx(g, 96, 512, hi=120)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    codes, scales = mp.moe_mxfp4_quantize(x, stream=side)
    eager = mp.moe_mxfp4_gemm(codes, scales, bc, bsc, stream=side)
    side.synchronize()
    gc, gs = torch.empty_like(codes), torch.empty_like(scales)
    go = torch.empty_like(eager)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mp.moe_mxfp4_quantize(x, gc, gs)
        mp.moe_mxfp4_gemm(gc, gs, bc, bsc, go)
    for i in range(4):
        x.copy_(torch.randn(50, 512, generator=g))
        graph.replay()
        want = mp.moe_mxfp4_gemm(*mp.moe_mxfp4_quantize(x), bc, bsc)
        torch.cuda.synchronize()
        assert torch.equal(go, want), i


@gpu
def test_binding_refusals_on_the_device():
    g = gen(11)
    a = [t.cuda() for t in random_mx(g, 4, 64)]
    b = [t.cuda() for t in random_mx(g, 2, 8, 64)]
    with pytest.raises(ValueError):
        mp.moe_mxfp4_gemm(*a, *b)                         # groups without bounds
    with pytest.raises(ValueError):
        mp.moe_mxfp4_gemm(*a, *b, bounds=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(TypeError):
        mp.moe_mxfp4_gemm(*a, *b, bounds=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        mp.moe_mxfp4_gemm(a[0], a[1], b[0][0, :, :16], b[1][0])      # another K
    with pytest.raises(ValueError):
        mp.moe_mxfp4_gemm(*a, b[0][0], b[1][0], out=torch.empty(3, 8, device="cuda"))
    with pytest.raises(ValueError):
        mp.moe_mxfp4_gemm(*a, b[0][0, :7].contiguous(), b[1][0, :7].contiguous(), swiglu=True)
    with pytest.raises(mp.MoePrefillError):
        mp.moe_mxfp4_quantize(torch.zeros(2, 48, device="cuda"))
    with pytest.raises((TypeError, ValueError)):
        mp.moe_mxfp4_quantize(torch.zeros(64, 4, device="cuda").t())
    with pytest.raises(TypeError):
        mp.moe_mxfp4_quantize(torch.zeros(2, 64, device="cuda", dtype=torch.float64))


@gpu
@pytest.mark.parametrize("swiglu", [False, True])
def test_many_empty_groups(swiglu):
    """More tile slots than a workgroup lists at a time, nearly all of groups without rows."""
    g = gen(11)
    G, M, N, K = 65535, 900, 150, 32
    ac, asc = random_mx(g, M, K, hi=120)
    bc, bsc = random_mx(g, G, 2 * N if swiglu else N, K, hi=120)
    held = sorted(torch.randperm(G, generator=g)[:12].tolist())
    held[0], held[-1] = 0, G - 1
    cuts = [0] + sorted(torch.randint(0, M + 1, (11,), generator=g).tolist()) + [M]
    bounds = torch.zeros(G + 1, dtype=torch.int32)
    for i, e in enumerate(held):
        bounds[e + 1:] = cuts[i + 1]
    out = torch.full((M, N), 77.0, device="cuda")
    mp.moe_mxfp4_gemm(ac.cuda(), asc.cuda(), bc.cuda(), bsc.cuda(), out, bounds=bounds.cuda(), swiglu=swiglu)
    want, err = ref.mx_product(ref.mx_values(ac, asc), ref.mx_values(bc[held], bsc[held]), torch.tensor(cuts), swiglu=swiglu)
    check_product(out, torch.float32, want, err)


@gpu
@pytest.mark.parametrize("far,M", [("a", 5), ("a just below", 130), ("a", 130), ("b", 3), ("b", 70), ("out", 70)])
def test_offsets_past_32_bits(far, M):
    """Codes of A (reached by a row table) or of B that span more than 2^32 bytes, or just fewer, and an
    output that does: all zero but for the rows that count."""
    g = gen(M)
    K = 64 if far == "out" else 1 << 18
    A = {"a": 32800, "a just below": 32767}.get(far, M)
    N = 33000 if far == "b" else 40
    a = [torch.zeros(A, K // 2, dtype=torch.uint8, device="cuda"), torch.full((A, K // 32), 127, dtype=torch.uint8, device="cuda")]
    b = [torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"), torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")]
    ar = sorted({0, A // 2, A - 2, A - 1}) if A > M else list(range(M))
    br = [0, N // 2, N - 1]
    for t, rows in ((a, ar), (b, br)):
        for m, v in zip(t, random_mx(g, len(rows), K, hi=118)):
            m[rows] = v.cuda()
    rows = torch.tensor(ar)[torch.randint(0, len(ar), (M,), generator=g)].int().cuda() if A > M else None
    stride = 1 << 26 if far == "out" else N
    buf = torch.empty((M - 1) * stride + N, device="cuda")
    out = buf.as_strided((M, N), (stride, 1))
    mp.moe_mxfp4_gemm(*a, *b, out, rows=rows)
    near = torch.searchsorted(torch.tensor(ar), rows.cpu().long()).int() if rows is not None else None
    want, err = ref.mx_product(ref.mx_values(a[0][ar], a[1][ar]), ref.mx_values(b[0][br], b[1][br])[None], rows=near)
    check_product(out[:, br], torch.float32, want, err)
    zero = torch.ones(N, dtype=torch.bool)
    zero[br] = False
    assert (out[:, zero.cuda()] == 0).all()


@gpu
def test_quantise_of_more_than_2_to_the_31_elements():
    M, K = 66000, 32768
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    codes, scales = mp.moe_mxfp4_quantize(x.fill_(1.5))
    for r0, r1 in ((0, 3), (40000, 40002), (M - 3, M)):
        assert (codes[r0:r1] == 0x77).all() and (scales[r0:r1] == 125).all()       # 1.5 = 6 * 2^-2
    tail = torch.randn(5, K, generator=gen(1)).bfloat16()
    x[-5:] = tail.cuda()
    mp.moe_mxfp4_quantize(x, codes, scales)
    check_quantised(tail, codes[-5:], scales[-5:], torch.bfloat16)
    back = mp.moe_mxfp4_dequantize(codes, scales, out=x)
    assert_same(back[-5:], ref.mx_values(codes[-5:], scales[-5:]).bfloat16())
    assert (back[:-5] == 1.5).all()


@gpu
def test_layer_of_the_operators_after_the_routing_of_a_prompt():
    """The products of a MoE layer on MXFP4 weights, with the row table, bounds and weights that the
    prompt path exports: quantise, gate/up with SwiGLU, quantise, down."""
    d, f, E, k, T = 256, 192, 10, 3, 150
    g = gen(5)
    R = T * k
    x = torch.randn(T, d, generator=g)
    logits = torch.randn(T, E, generator=g)
    logits[:, 7] = -50.0                                  # an expert without rows
    wgu = mp.moe_mxfp4_quantize((torch.randn(E * 2 * f, d, generator=g) / 16).cuda())
    wd = mp.moe_mxfp4_quantize((torch.randn(E * d, f, generator=g) / 16).cuda())
    wgu, wd = [t.view(E, 2 * f, -1) for t in wgu], [t.view(E, d, -1) for t in wd]
    ex = dict(rows=torch.empty(R, dtype=torch.int32, device="cuda"), bounds=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
              weights=torch.empty(T, k, device="cuda"))
    h = mp.moe_prefill_create(d, f, E, k, T)
    blob = torch.zeros(mp.moe_prefill_layer_bytes(d, f, E), dtype=torch.uint8, device="cuda")
    y = torch.empty(T, d, device="cuda")
    mp.moe_prefill_run_layer(h, x.cuda(), logits.cuda(), y, weights=blob, exports=ex)
    xq = mp.moe_mxfp4_quantize(x.cuda())
    hh = mp.moe_mxfp4_gemm(*xq, *wgu, bounds=ex["bounds"], rows=ex["rows"], top_k=k, swiglu=True, dtype=torch.bfloat16)
    hq = mp.moe_mxfp4_quantize(hh)
    dm = mp.moe_mxfp4_gemm(*hq, *wd, bounds=ex["bounds"])
    pair = ex["rows"].long()
    y.zero_().index_add_(0, pair // k, dm * ex["weights"].view(-1)[pair, None])
    torch.cuda.synchronize()
    h.close()
    bounds, rows = ex["bounds"].cpu(), ex["rows"].cpu()
    assert bounds[0] == 0 and bounds[-1] == R and bounds[7] == bounds[8]
    want, err = ref.mx_product(ref.mx_values(*xq), ref.mx_values(*wgu), bounds, rows, k, True)
    check_product(hh, torch.bfloat16, want, err)
    check_quantised(hh, *hq, torch.bfloat16)
    want, err = ref.mx_product(ref.mx_values(*hq), ref.mx_values(*wd), bounds, torch.arange(R).int(), 1)
    check_product(dm, torch.float32, want, err)
    # by the dense formula: the 4-bit roundings of x, h and both weights (an element of a block of 32
    # normal values is off by about a tenth of its rms) make it a fifth to a third of the output's norm
    full, wg, wdn = torch.zeros(T, d, dtype=torch.float64), ref.mx_values(*wgu), ref.mx_values(*wd)
    wt = torch.softmax(logits.double().topk(k, -1).values, -1)
    for t in range(T):
        for j, e in enumerate(logits[t].topk(k).indices.tolist()):
            z = wg[e] @ x[t].double()
            full[t] += wt[t, j] * (wdn[e] @ (z[:f] * torch.sigmoid(z[:f]) * z[f:]))
    assert float((y.cpu() - full).norm() / full.norm()) < 0.4


@gpu
def test_products_on_two_streams_at_once():
    g = gen(6)
    sets = []
    for M, N, K in ((700, 900, 1024), (2500, 4200, 512)):
        a, b = ([t.cuda() for t in random_mx(g, n, K)] for n in (M, N))
        sets.append((a, b, mp.moe_mxfp4_gemm(*a, *b)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(4):
        for (a, b, want), s in zip(sets, streams):
            o = torch.full_like(want, 77.0)
            s.wait_stream(torch.cuda.current_stream())
            mp.moe_mxfp4_gemm(*a, *b, o, stream=s)
            outs.append((o, want))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in outs)
