"""Plain 64-bit forms of the MXFP4 operators and of the few-token layer, written from the
formulas, with the error bounds that the tests hold the kernels to."""
from __future__ import annotations

import math

import torch

MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def half_step(dtype) -> float:
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def least_step(dtype) -> float:
    """Half the distance of dtype's smallest numbers: the absolute error of a rounding below its
    normal range.  fp16 reaches 2^-24, so 2^-25; fp32's and bf16's lie below every value here."""
    return 2.0 ** -25 if dtype == torch.float16 else 0.0


def mx_quantize(x: torch.Tensor):
    """x [M, K] (any float type) -> (codes [M, K/2], scales [M, K/32]) uint8, element by element
    against the eight magnitudes: the nearest, ties to the even code."""
    v = x.double().cpu().reshape(x.shape[0], -1, 32)
    bad = ~torch.isfinite(v).all(-1)
    v = torch.where(bad[..., None], torch.zeros_like(v), v)
    amax = v.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full(amax.shape, -127)).clamp(min=-127)
    q = torch.ldexp(v.abs(), -e[..., None])
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64)
    dist = (q[..., None] - mags).abs()
    # a tie is between neighbours: prefer the even code
    dist = dist + torch.tensor([0.0, 1e-9] * 4, dtype=torch.float64)
    code = dist.argmin(-1) + 8 * torch.signbit(v)
    code = torch.where(bad[..., None], torch.zeros_like(code), code).reshape(x.shape[0], -1, 2)
    scales = torch.where(bad, torch.full_like(e, 255), e + 127)
    return (code[..., 0] | (code[..., 1] << 4)).to(torch.uint8), scales.to(torch.uint8)


def mx_values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """[..., K/2] codes and [..., K/32] scale bytes -> fp64 values [..., K]."""
    codes, scales = codes.cpu(), scales.cpu()
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), dtype=torch.float64)
    v = table[torch.stack([codes & 15, codes >> 4], -1).long()].reshape(*codes.shape[:-1], -1)
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return v * s.repeat_interleave(32, -1)


def mx_product(a, b, bounds=None, rows=None, top_k=1, swiglu=False):
    """a [A, K], b [G, NB, K] fp64 -> (out [M, N] fp64, bound on an fp32 evaluation's error), NaN
    rows where no group holds the row.  Bound: every one of the K additions of a sum is off by at
    most 2^-23 of the sum of magnitudes (a rounding or a truncation to 24 bits)."""
    M = rows.numel() if rows is not None else a.shape[0] * top_k
    src = (rows.cpu().long() if rows is not None else torch.arange(M)) // top_k
    NB = b.shape[1]
    src = src.to(a.device)
    z = torch.full((M, NB), math.nan, dtype=torch.float64, device=a.device)
    mag = torch.full_like(z, math.nan)
    edges = bounds.tolist() if bounds is not None else [0, M]
    for g, (lo, hi) in enumerate(zip(edges, edges[1:])):
        if hi > lo:
            z[lo:hi] = a[src[lo:hi]] @ b[g].t()
            mag[lo:hi] = a[src[lo:hi]].abs() @ b[g].abs().t()
    err = a.shape[1] * 2.0 ** -23 * mag
    if not swiglu:
        return z, err
    g, u = z[:, : NB // 2], z[:, NB // 2:]
    return _swiglu(g, u, err[:, : NB // 2], err[:, NB // 2:])


def _swiglu(g, u, eg, eu):
    """silu(g) u and its error from errors of g and u: |silu'| <= 1.1, the fp32 exponential,
    sum, division and product add at most 8 half steps; exp(-g) of an off g is in eg."""
    s = g * torch.sigmoid(g)
    h = s * u
    return h, 1.1 * eg * (u.abs() + eu) + s.abs() * eu + 8 * 2.0 ** -24 * h.abs()


def layer(x, logits, k, gu_q, gu_s, d_q, d_s):
    """The few-token layer in fp64: x [T, d], logits [T, E], codes and fp16 scales of the experts.
    Returns (y, bound on |kernel - y| before the rounding to the output's type, eidx, weights).

    The bound: a block of 32 activations in fixed point is off by 2^-23 (1 + 1/64) of its largest
    magnitude (24 bits, for fp32 x) or 2^-15 (1 + 1/64) (16 bits, for bf16 and fp16); a sum over nb blocks in fp32 makes at most nb + 6 roundings of 2^-24 of the sum of
    magnitudes (join, scale product and fma per block, then the waves' sums); the router weights
    are off by k + 8 half steps and the combine by k."""
    step = 2.0 ** -23 if x.dtype == torch.float32 else 2.0 ** -15
    x, logits = x.double().cpu(), logits.double().cpu()
    T, E = logits.shape
    d, f = x.shape[1], gu_q.shape[1] // 2
    y = torch.zeros(T, d, dtype=torch.float64)
    bound = torch.zeros_like(y)
    eidx = torch.full((T, k), -1, dtype=torch.int32)
    wts = torch.zeros(T, k, dtype=torch.float64)

    def product(v, ev, q, s):
        w = q.double().cpu() * s.double().cpu().repeat_interleave(32, -1)
        nb = v.numel() // 32
        fixed = v.reshape(nb, 32).abs().amax(-1).repeat_interleave(32) * step * (1 + 1 / 64)
        err = w.abs() @ (ev + fixed) + 2 * (nb + 6) * 2.0 ** -24 * (w.abs() @ v.abs())
        return w @ v, err

    for t in range(T):
        order = sorted(range(E), key=lambda e: (-float(logits[t, e]), e))[:k]
        live = [e for e in order if float(logits[t, e]) > -math.inf]
        if not live:
            continue
        z = torch.exp(logits[t, live] - logits[t, live[0]])
        w = z / z.sum()
        for j, e in enumerate(live):
            eidx[t, j], wts[t, j] = e, w[j]
            zz, ez = product(x[t], torch.zeros(d, dtype=torch.float64), gu_q[e], gu_s[e])
            h, eh = _swiglu(zz[:f], zz[f:], ez[:f], ez[f:])
            dm, edm = product(h, eh, d_q[e], d_s[e])
            y[t] += w[j] * dm
            bound[t] += w[j] * edm + (2 * k + 8) * 2.0 ** -24 * w[j] * (dm.abs() + edm)
    return y, bound, eidx, wts
