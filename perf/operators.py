"""Measured cases of the few-token MoE layer and of the MXFP4 operators.

Three operators, each in its plain form (elementary torch operations in fp32) and
as a user calls the framework's entry points (`own`):

  layer     one MoE FFN layer for a few tokens (`moe_decode_run_layer`): top-k of the
            router logits, softmax over the k selected, per expert
            h = silu(x Wg^T) * (x Wu^T), y = sum_j w_j h_j Wd^T, the weights in the
            packed Q4 layer blob of the prompt path, the activations not quantised
  quantise  a matrix to MXFP4 (`moe_mxfp4_quantize`) and back (`moe_mxfp4_dequantize`)
  product   Y = A B^T of two MXFP4 matrices (`moe_mxfp4_gemm`): one weight matrix, or
            one per expert over the groups of the router's row table, with gathered
            rows and SwiGLU in the same call where the case says so

MXFP4: blocks of 32 along K, one power-of-two scale 2^(s - 127) (E8M0 byte s) per
block, elements E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), two to a byte,
the lower index in the low nibble.  Scale of a block: floor(log2(max |x|)) - 2.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32
_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # one user's next token through a layer of the resident configuration: latency
        dict(name="layer 1 token", op="layer", T=1, d=2048, f=768, E=128, k=8, dtype="bf16", skew=0.0, idle=0, pad=0),
        # a handful of users, or the drafted tokens of one, kept in fp32
        dict(name="layer 5 tokens f32", op="layer", T=5, d=2048, f=768, E=128, k=8, dtype="f32", skew=0.0, idle=0, pad=0),
        # the wide layer of the largest configuration, one token: the weights' bytes
        dict(name="layer 1 token wide", op="layer", T=1, d=4096, f=1536, E=256, k=8, dtype="f32", skew=0.0, idle=0, pad=0),
        # a serving batch on the wide layer under its skewed routing, two slots of the batch empty
        dict(name="layer 24 tokens wide", op="layer", T=24, d=4096, f=1536, E=256, k=8, dtype="bf16", skew=1.1, idle=2, pad=0),
        # odd sizes: half K pairs, an expert count that is no power of two, rows of a wider buffer
        dict(name="layer 3 tokens odd", op="layer", T=3, d=1184, f=352, E=60, k=4, dtype="f16", skew=0.5, idle=0, pad=24),
        # one token's activations before a product: latency
        dict(name="quantise 1 row", op="quantise", M=1, K=2048, dtype="bf16", pad=0),
        # a prompt's activations at the widest model, fp32 as the layer takes them
        dict(name="quantise 8192 rows f32", op="quantise", M=8192, K=4096, dtype="f32", pad=0),
        # a ragged prompt whose rows lie in a wider buffer
        dict(name="quantise 1333 rows f16", op="quantise", M=1333, K=1504, dtype="f16", pad=40),
        # a single token through one weight matrix, its activations quantised on the way
        dict(name="product 1 row", op="product", M=1, N=4096, K=4096, E=0, k=1, dtype="bf16", quantise=True, swiglu=False, skew=0.0),
        # a whole prompt through one weight matrix: the matrix cores' rate
        dict(name="product 8192 rows", op="product", M=8192, N=4096, K=4096, E=0, k=1, dtype="bf16", quantise=False, swiglu=False, skew=0.0),
        # gate and up of the resident configuration: rows gathered for 128 experts, SwiGLU in the call
        dict(name="experts gate up 1024 tokens", op="product", M=1024, N=768, K=2048, E=128, k=8, dtype="bf16", quantise=True, swiglu=True, skew=0.0),
        # the down product of the wide layer over a skewed row table
        dict(name="experts down 24576 rows", op="product", M=24576, N=4096, K=1536, E=256, k=1, dtype="f32", quantise=False, swiglu=False, skew=0.5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer", "layer", "quantise", "product", "product"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "layer":
        E = rng.randint(4, 200)
        return dict(op=op, T=_log_int(rng, 1, 24), d=32 * _log_int(rng, 4, 128), f=32 * _log_int(rng, 2, 48), E=E,
                    k=rng.randint(1, min(8, E)), dtype=dtype, skew=rng.choice([0.0, 0.5, 1.1]), idle=rng.choice([0, 0, 1]),
                    pad=8 * rng.randint(0, 6))
    if op == "quantise":
        return dict(op=op, M=_log_int(rng, 1, 8000), K=32 * _log_int(rng, 1, 128), dtype=dtype, pad=8 * rng.randint(0, 6))
    E = rng.choice([0, 0, rng.randint(2, 160)])
    k = rng.randint(1, min(8, E)) if E else 1
    swiglu = rng.random() < 0.4
    return dict(op=op, M=_log_int(rng, 1, 8000 if not E else max(1, 12000 // k)), N=_log_int(rng, 16, 2048 if E or swiglu else 4096),
                K=32 * _log_int(rng, 1, 128 if not E else 64), E=E, k=k, dtype=dtype, quantise=rng.random() < 0.5,
                swiglu=swiglu, skew=rng.choice([0.0, 0.5]))


# ----------------------------------------------------------------- inputs ---

def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed) * 1000003 + 17)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=_dev(), dtype=torch.float32)


def _rows(x, dtype, pad):
    """x [M, K] in `dtype`, its rows in a buffer of K + pad columns."""
    buf = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=_DTYPES[dtype], device=x.device)
    buf[:, : x.shape[1]] = x
    return buf[:, : x.shape[1]]


def _logits(g, T, E, skew, idle):
    lg = _normal(g, T, E)
    if skew:                                    # popularity of a Zipf(skew) expert ranking
        rank = torch.randperm(E, generator=g, device=lg.device).float() + 1
        lg -= skew * rank.log()
    if idle:                                    # empty slots of a padded batch: no expert allowed
        lg[T - min(idle, T):] = -math.inf
    return lg


def _pad_last(x, to, value):
    return x if x.shape[-1] == to else torch.nn.functional.pad(x, (0, to - x.shape[-1]), value=value)


def _tile_codes(q):
    """Codes [E, N, K] int8 in [-8, 7] -> the blob's 32-row tiles by K pairs, [E, bytes]."""
    E, N, K = q.shape
    K64 = -(-K // 64) * 64
    u = _pad_last((q + 8).to(torch.uint8), K64, 8).view(E, N // 32, 32, K64 // 64, 2, 2, 2, 2, 4)
    b = u[..., 0, :] | (u[..., 1, :] << 4)      # [E, tile, row, pair, block, half, word, byte]
    return b.permute(0, 1, 3, 5, 2, 4, 6, 7).reshape(E, -1)


def _tile_scales(s):
    """Scales [E, N, K / 32] fp16 -> groups of 8 blocks a row, [E, bytes]."""
    E, N, nb = s.shape
    nb8 = -(-nb // 8) * 8
    s = _pad_last(s, nb8, 0.0).view(E, N // 32, 32, nb8 // 8, 8).permute(0, 1, 3, 2, 4)
    return s.reshape(E, -1).contiguous().view(torch.uint8)


def _blob(gu_q, gu_s, d_q, d_s):
    """The packed layer blob: per expert gate/up codes and scales (gate and up tiles in
    turn), down codes and scales, each section 256-byte aligned."""
    E, f2, d = gu_q.shape
    f = f2 // 2
    turn = lambda w: w.view(E, 2, f // 32, 32, -1).transpose(1, 2).reshape(E, f2, -1)  # noqa: E731
    parts = [_tile_codes(turn(gu_q)), _tile_scales(turn(gu_s)), _tile_codes(d_q), _tile_scales(d_s)]
    return torch.cat([_pad_last(p, -(-p.shape[1] // 256) * 256, 0) for p in parts], 1).reshape(-1)


def _prepare_layer(c, g):
    T, d, f, E, k = c["T"], c["d"], c["f"], c["E"], c["k"]

    def codes(*shape):
        return torch.randint(-8, 8, shape, generator=g, device=_dev(), dtype=torch.int8)

    def scales(rows, n_in):
        u = torch.rand(E, rows, n_in // 32, generator=g, device=_dev())
        return ((0.5 + u) / math.sqrt(n_in)).half()

    gu_q, gu_s = codes(E, 2 * f, d), scales(2 * f, d)
    d_q, d_s = codes(E, d, f), scales(d, f)
    s = dict(x=_rows(_normal(g, T, d), c["dtype"], c["pad"]), logits=_logits(g, T, E, c["skew"], c["idle"]),
             gu_q=gu_q, gu_s=gu_s, d_q=d_q, d_s=d_s, blob=_blob(gu_q, gu_s, d_q, d_s))
    s["y"] = _rows(torch.zeros(T, d, device=_dev()), c["dtype"], c["pad"])
    if own:
        import moe_prefill_ffn_amd as mp

        s["handle"] = mp.moe_prefill_create(d, f, E, k, T, device=_dev().index)
        s["workspace"] = torch.empty(mp.moe_decode_workspace_size(d, f, E, k, T), dtype=torch.uint8, device=_dev())
    return s


def _mx_random(g, *shape):
    """A random MXFP4 matrix [..., K]: packed codes and scale bytes of weight-like size."""
    K = shape[-1]
    codes = torch.randint(0, 256, (*shape[:-1], K // 2), generator=g, device=_dev(), dtype=torch.uint8)
    scales = torch.randint(112, 124, (*shape[:-1], K // BLOCK), generator=g, device=_dev(), dtype=torch.uint8)
    return codes, scales


def _prepare_product(c, g):
    M, N, K, E, k = c["M"], c["N"], c["K"], c["E"], c["k"]
    s = dict(out=torch.zeros(M * k, N, dtype=_DTYPES[c["dtype"]], device=_dev()))
    wide = 2 * N if c["swiglu"] else N
    s["b_codes"], s["b_scales"] = _mx_random(g, E or 1, wide, K)
    if c["quantise"]:
        s["x"] = _normal(g, M, K).to(_DTYPES["f32" if c["dtype"] == "f32" else "bf16"])
        s["a_codes"] = torch.empty(M, K // 2, dtype=torch.uint8, device=_dev())
        s["a_scales"] = torch.empty(M, K // BLOCK, dtype=torch.uint8, device=_dev())
    else:
        s["a_codes"], s["a_scales"] = _mx_random(g, M, K)
    if E:                                       # the row table: pairs p = t * k + j grouped by expert
        chosen = torch.topk(_logits(g, M, E, c["skew"], 0), k).indices.reshape(-1)
        s["rows"] = torch.sort(chosen, stable=True).indices.int()
        counts = torch.bincount(chosen, minlength=E)
        s["bounds"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        s["splits"] = counts.tolist()           # rows of each group, known to who made the table
        if k == 1 and not c["quantise"]:        # rows that stand in the table's order already
            s["rows"] = None
    return s


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    if c["op"] == "layer":
        s = _prepare_layer(c, g)
    elif c["op"] == "quantise":
        s = dict(x=_rows(_normal(g, c["M"], c["K"]) * torch.exp(_normal(g, c["M"], 1)), c["dtype"], c["pad"]))
        s["codes"] = torch.empty(c["M"], c["K"] // 2, dtype=torch.uint8, device=_dev())
        s["scales"] = torch.empty(c["M"], c["K"] // BLOCK, dtype=torch.uint8, device=_dev())
        s["values"] = torch.empty(c["M"], c["K"], dtype=_DTYPES[c["dtype"]], device=_dev())
    else:
        s = _prepare_product(c, g)
    s["case"] = c
    return s


# ------------------------------------------------------------ plain forms ---

def _pow2(byte):
    """2^(byte - 127) in fp32, exactly (byte 0 is the subnormal 2^-127)."""
    i = byte.to(torch.int32)
    return torch.where(i == 0, torch.full_like(i, 0x00400000), i << 23).view(torch.float32)


def _mx_values(codes, scales):
    lut = torch.tensor(_E2M1, dtype=torch.float32, device=codes.device)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1)
    v = v.reshape(*scales.shape, BLOCK)
    return (v * _pow2(scales)[..., None]).reshape(*codes.shape[:-1], -1)


def _mx_quantise(x):
    """Packed codes and scale bytes of x [M, K]: scale 2^(floor(log2(amax)) - 2), elements
    to the nearest of the eight magnitudes, ties to the even code, 6 beyond the largest."""
    b = x.float().reshape(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1)
    byte = ((amax.view(torch.int32) >> 23) - 2).clamp(min=0)
    a = b.abs() / _pow2(byte)[..., None]
    # steps of 0.5 below 2, of 1 below 4, of 2 above: the code is the rounded count of steps
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    base = torch.where(a < 2, 0.0, torch.where(a < 4, 2.0, 4.0))
    code = (torch.round(a / step) + base).clamp(max=7).to(torch.uint8) | (torch.signbit(b).to(torch.uint8) << 3)
    code = code.reshape(x.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), byte.to(torch.uint8)


def _plain_layer(s):
    c, x, lg = s["case"], s["x"].float(), s["logits"]
    k, E, d, f = c["k"], c["E"], c["d"], c["f"]
    order = torch.sort(lg, dim=-1, descending=True, stable=True)          # ties: the lower expert
    top, idx = order.values[:, :k], order.indices[:, :k].reshape(-1)
    e = torch.exp(top - torch.where(top[:, :1] == -math.inf, 0.0, top[:, :1]))
    w = e / e.sum(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).tiny)   # no expert allowed: all weights 0
    used, slot = torch.unique(idx, return_inverse=True)

    def weights(q, sc):
        return q[used].float().view(used.numel(), q.shape[1], -1, BLOCK) * sc[used].float()[..., None]

    gu = weights(s["gu_q"], s["gu_s"]).view(-1, 2 * f, d)
    xp = x.repeat_interleave(k, 0)                                    # one row per (token, slot)
    per = torch.bincount(slot, minlength=used.numel())
    place = torch.argsort(slot, stable=True)
    first = per.cumsum(0) - per
    col = torch.arange(idx.numel(), device=x.device) - first[slot[place]]
    cap = c["T"] if c["T"] < 64 else int(per.max())
    a = x.new_zeros(used.numel(), cap, d)
    a[slot[place], col] = xp[place]
    z = torch.bmm(a, gu.transpose(1, 2).contiguous())
    del gu
    h = z[..., :f] / (1 + torch.exp(-z[..., :f])) * z[..., f:]
    dm = torch.bmm(h, weights(s["d_q"], s["d_s"]).view(-1, d, f).transpose(1, 2).contiguous())
    rows = torch.empty_like(xp)
    rows[place] = dm[slot[place], col]
    y = (rows.view(-1, k, d) * w[..., None]).sum(1)
    return y.to(_DTYPES[c["dtype"]])


def _plain_product(s):
    c = s["case"]
    codes, scales = _mx_quantise(s["x"]) if c["quantise"] else (s["a_codes"], s["a_scales"])
    a, b = _mx_values(codes, scales), _mx_values(s["b_codes"], s["b_scales"])
    if c["E"]:
        if s["rows"] is not None:
            a = a[(s["rows"] // c["k"]).long()]
        z = torch.cat([rows @ w.t() for rows, w in zip(a.split(s["splits"]), b)])
    else:
        z = a @ b[0].t()
    if c["swiglu"]:
        gate, up = z[:, : c["N"]], z[:, c["N"]:]
        z = gate / (1 + torch.exp(-gate)) * up
    return z.to(_DTYPES[c["dtype"]])


# -------------------------------------------------------------------- run ---

def _own(s):
    import moe_prefill_ffn_amd as mp

    c = s["case"]
    if c["op"] == "layer":
        mp.moe_decode_run_layer(s["handle"], s["x"], s["logits"], s["y"], weights=s["blob"], workspace=s["workspace"])
        return s["y"]
    if c["op"] == "quantise":
        mp.moe_mxfp4_quantize(s["x"], s["codes"], s["scales"])
        mp.moe_mxfp4_dequantize(s["codes"], s["scales"], s["values"])
        return {"values": s["values"], "scales": s["scales"]}
    if c["quantise"]:
        mp.moe_mxfp4_quantize(s["x"], s["a_codes"], s["a_scales"])
    mp.moe_mxfp4_gemm(s["a_codes"], s["a_scales"], s["b_codes"], s["b_scales"], s["out"], bounds=s.get("bounds"),
                      rows=s.get("rows"), top_k=c["k"], swiglu=c["swiglu"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op == "layer":
        return _plain_layer(state)
    if op == "quantise":
        codes, scales = _mx_quantise(state["x"])
        return {"values": _mx_values(codes, scales).to(state["values"].dtype), "scales": scales}
    return _plain_product(state)


# ------------------------------------------------------------------- work ---

def work(case):
    c = case
    if c["op"] == "layer":
        live = max(0, c["T"] - c["idle"])
        pairs = live * c["k"]
        # experts that some row of evenly spread routing reaches; skew reaches fewer
        reached = c["E"] * (1 - (1 - c["k"] / c["E"]) ** live)
        weights = 3 * c["d"] * c["f"]
        return {"bytes": reached * weights * (0.5 + 2 / 32) + c["T"] * (c["d"] * 2 * _BYTES[c["dtype"]] + 4 * c["E"]),
                "flops": 2.0 * pairs * weights}
    if c["op"] == "quantise":
        n = c["M"] * c["K"]
        return {"bytes": n * 2 * _BYTES[c["dtype"]] + 2 * n * (0.5 + 1 / 32), "flops": 4.0 * n}
    rows, wide = c["M"] * c["k"], c["N"] * (2 if c["swiglu"] else 1)
    groups = c["E"] * (1 - (1 - 1 / c["E"]) ** rows) if c["E"] else 1
    mx = 0.5 + 1 / 32
    a_bytes = c["M"] * c["K"] * (mx + ((4 if c["dtype"] == "f32" else 2) + mx if c["quantise"] else 0))
    return {"bytes": a_bytes + groups * wide * c["K"] * mx + rows * c["N"] * _BYTES[c["dtype"]], "flops": 2.0 * rows * wide * c["K"]}


# ------------------------------------------------------- 64-bit definition ---

def _exact_mx(x):
    """x [M, K] rounded to MXFP4, as fp64 values and the scale bytes."""
    b = x.double().view(x.shape[0], -1, BLOCK)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 1 - 2, -127).clamp(min=-127)
    q = b / torch.exp2(e.double())[..., None]
    m = torch.frexp(q).exponent.clamp(min=1, max=3) - 2                 # exponent of the element's last place: 2^m
    step = torch.exp2(m.double())
    v = (torch.round(q / step) * step).clamp(-6, 6)
    return (v * torch.exp2(e.double())[..., None]).view(x.shape), (e + 127).to(torch.uint8)


def _exact_values(codes, scales):
    nib = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).long()
    mag, ex = (nib & 1).double(), (nib >> 1) & 3
    v = torch.where(ex == 0, mag * 0.5, (1 + mag * 0.5) * torch.exp2((ex - 1).double()))
    v = torch.where(nib >= 8, -v, v)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "quantise":
        values, scales = _exact_mx(s["x"])
        return {"values": values, "scales": scales}
    if c["op"] == "layer":
        f, k = c["f"], c["k"]
        y = torch.zeros(c["T"], c["d"], dtype=torch.float64, device=_dev())
        w64 = lambda q, sc: q.double() * sc.double().repeat_interleave(BLOCK, -1)  # noqa: E731
        order = sorted
        for t in range(c["T"]):
            lg = s["logits"][t].double().tolist()
            best = order(range(c["E"]), key=lambda e: (-lg[e], e))[:k]
            best = [e for e in best if lg[e] > -math.inf]
            total = sum(math.exp(lg[e] - lg[best[0]]) for e in best)
            for e in best:
                z = w64(s["gu_q"][e], s["gu_s"][e]) @ s["x"][t].double()
                h = z[:f] * torch.sigmoid(z[:f]) * z[f:]
                y[t] += math.exp(lg[e] - lg[best[0]]) / total * (w64(s["d_q"][e], s["d_s"][e]) @ h)
        return y
    a = _exact_mx(s["x"])[0] if c["quantise"] else _exact_values(s["a_codes"], s["a_scales"])
    groups = s["bounds"].tolist() if c["E"] else [0, c["M"]]
    rows = s.get("rows")
    a = a[torch.div(rows, c["k"], rounding_mode="floor").long()] if rows is not None else a
    parts = [a[lo:hi] @ _exact_values(s["b_codes"][e], s["b_scales"][e]).t()
             for e, (lo, hi) in enumerate(zip(groups, groups[1:])) if hi > lo]
    z = torch.cat(parts)
    if c["swiglu"]:
        z = z[:, : c["N"]] * torch.sigmoid(z[:, : c["N"]]) * z[:, c["N"]:]
    return z
