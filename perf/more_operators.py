"""Measured cases of the 16-bit experts' operators and of the low-rank adapters.

Four operators, each in its plain form (elementary torch operations in fp32) and as a
user calls the framework's entry points (`own`):

  group     the row table of any routing (`moe_group_rows`): pairs p = t * k + j ordered
            by their expert, each expert's bounds, and every pair's place; a pair whose
            expert is -1 (an empty slot of a padded batch) is in no group
  product   out[r] = A[src(r)] B[g(r)]^T of 16-bit matrices (`moe_grouped_gemm`): one
            weight matrix, or one per expert over the groups of a row table, with
            gathered rows and SwiGLU in the same call where the case says so
  combine   y[t] = base[t] + sum_j w[t, j] D[pos[t, j]] (`moe_combine_rows`): the experts'
            rows back to tokens, added to the output of a shared expert
  lora      out[t] = base[t] + s_i (x[t] A_i^T) B_i^T with i the adapter of row t
            (`moe_lora_add`): the adapters of many requests beside a shared projection,
            whose output is `base`
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------ cases ---

def listed():
    return [
        # a serving batch's routing on the wide layer, two slots of the batch empty: latency
        dict(name="group 24 tokens", op="group", T=24, E=256, k=8, skew=1.1, idle=2),
        # the largest prompt's routing under its skew
        dict(name="group 8192 tokens", op="group", T=8192, E=256, k=8, skew=1.1, idle=0),
        # gate and up of one user's next token through 16-bit experts: eight experts' bytes
        dict(name="experts gate up 1 token", op="product", M=1, N=768, K=2048, E=128, k=8, dtype="bf16", out="bf16", swiglu=True, skew=0.0, pad=0),
        # a prompt of the resident configuration: 64 rows an expert, the weights' bytes
        dict(name="experts gate up 1024 tokens", op="product", M=1024, N=768, K=2048, E=128, k=8, dtype="bf16", out="bf16", swiglu=True, skew=0.0, pad=0),
        # down of the largest prompt, rows that stand in the table's order: 256 rows an expert and skewed
        dict(name="experts down 65536 rows", op="product", M=65536, N=4096, K=1536, E=256, k=1, dtype="bf16", out="bf16", swiglu=False, skew=0.5, pad=0),
        # the largest prompt through one shared matrix: the matrix cores' rate
        dict(name="shared projection 8192 rows", op="product", M=8192, N=4096, K=4096, E=0, k=1, dtype="bf16", out="bf16", swiglu=False, skew=0.0, pad=0),
        # odd sizes: K that ends inside a tile, an odd N, rows of a wider buffer, fp32 out
        dict(name="experts 333 tokens odd", op="product", M=333, N=1001, K=1192, E=60, k=4, dtype="f16", out="f32", swiglu=False, skew=0.5, pad=24),
        # the experts' rows of a few drafted tokens: latency
        dict(name="combine 5 tokens f32", op="combine", T=5, d=2048, k=8, dtype="f32", out="f32", idle=1, pad=0),
        # the largest prompt, beside a shared expert's output: memory
        dict(name="combine 8192 tokens", op="combine", T=8192, d=4096, k=8, dtype="bf16", out="bf16", idle=0, pad=0),
        # one user's next token with an adapter: latency
        dict(name="adapters 1 row", op="lora", M=1, K=4096, N=4096, r=16, n=4, runs=1, none=0.0, dtype="bf16", base="bf16", out="bf16", pad=0),
        # a serving batch, every row another request's, some without an adapter; odd sizes, rows of a wider buffer
        dict(name="adapters 48 rows mixed", op="lora", M=48, K=1184, N=2051, r=24, n=30, runs=48, none=0.2, dtype="f16", base="f32", out="f32", pad=8),
        # the prompts of eight requests in one batch
        dict(name="adapters 8192 rows", op="lora", M=8192, K=4096, N=4096, r=64, n=8, runs=8, none=0.1, dtype="bf16", base="bf16", out="bf16", pad=0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["group", "product", "product", "product", "combine", "lora", "lora"])
    dtype = rng.choice(["bf16", "f16"])
    if op == "group":
        E = _log_int(rng, 2, 512)
        return dict(op=op, T=_log_int(rng, 1, 16000), E=E, k=rng.randint(1, min(8, E)), skew=rng.choice([0.0, 0.5, 1.1]),
                    idle=rng.choice([0, 1, 3]))
    if op == "product":
        E = rng.choice([0, 0, rng.randint(2, 160)])
        k = rng.randint(1, min(8, E)) if E else 1
        swiglu = rng.random() < 0.4
        return dict(op=op, M=_log_int(rng, 1, 8000 if not E else 16000 // k), N=_log_int(rng, 16, 2048 if E or swiglu else 4096),
                    K=8 * _log_int(rng, 4, 256 if E else 512), E=E, k=k, dtype=dtype, out=rng.choice(["f32", dtype]), swiglu=swiglu,
                    skew=rng.choice([0.0, 0.5]), pad=8 * rng.randint(0, 6))
    if op == "combine":
        return dict(op=op, T=_log_int(rng, 1, 8000), d=_log_int(rng, 8, 512) * rng.choice([1, 8]), k=rng.randint(1, 8),
                    dtype=rng.choice(["f32", dtype]), out=rng.choice(["f32", dtype]), idle=rng.choice([0, 1]), pad=8 * rng.randint(0, 6))
    M, n = _log_int(rng, 1, 8000), _log_int(rng, 1, 48)
    out = rng.choice(["f32", dtype])
    return dict(op=op, M=M, K=8 * _log_int(rng, 8, 512), N=_log_int(rng, 32, 4096), r=8 * _log_int(rng, 1, 16), n=n,
                runs=min(M, rng.choice([1, n, 2 * n, M if M <= 512 else n])), none=rng.choice([0.0, 0.2]), dtype=dtype,
                base=rng.choice(["f32", out]), out=out, pad=8 * rng.randint(0, 6))


# ----------------------------------------------------------------- inputs ---

def _dev():
    return torch.device("cuda", torch.cuda.current_device())


def _gen(seed):
    g = torch.Generator(device=_dev())
    g.manual_seed(int(seed) * 1000003 + 29)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=_dev(), dtype=torch.float32)


def _rows(x, dtype, pad):
    """x [M, K] in `dtype`, its rows in a buffer of K + pad columns."""
    buf = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=_DTYPES[dtype], device=x.device)
    buf[:, : x.shape[1]] = x
    return buf[:, : x.shape[1]]


def _weights(g, dtype, *shape):
    """Matrices [G, N, K] of weight-like size, made a slice at a time."""
    w = torch.empty(*shape, dtype=_DTYPES[dtype], device=_dev())
    for i in range(shape[0]):
        w[i] = _normal(g, *shape[1:]) / math.sqrt(shape[-1])
    return w


def _chosen(g, T, E, k, skew):
    """The experts of T tokens, [T, k], by a router whose experts have a Zipf(skew) popularity."""
    lg = _normal(g, T, E)
    if skew:
        rank = torch.randperm(E, generator=g, device=lg.device).float() + 1
        lg -= skew * rank.log()
    return torch.topk(lg, k).indices.int()


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    s = dict(case=c)
    if c["op"] == "group":
        T, P = c["T"], c["T"] * c["k"]
        s["eidx"] = _chosen(g, T, c["E"], c["k"], c["skew"])
        if c["idle"]:
            s["eidx"][T - min(c["idle"], T):] = -1
        s["bounds"] = torch.zeros(c["E"] + 1, dtype=torch.int32, device=_dev())
        s["rows"] = torch.zeros(P, dtype=torch.int32, device=_dev())
        s["pos"] = torch.zeros(T, c["k"], dtype=torch.int32, device=_dev())
        if own:
            import moe_prefill_ffn_amd as mp

            s["workspace"] = torch.empty(mp.moe_group_workspace_size(P, c["E"]), dtype=torch.uint8, device=_dev())
    elif c["op"] == "product":
        M, N, K, E, k = c["M"], c["N"], c["K"], c["E"], c["k"]
        s["a"] = _rows(_normal(g, M, K), c["dtype"], c["pad"])
        s["b"] = _weights(g, c["dtype"], E or 1, 2 * N if c["swiglu"] else N, K)
        s["out"] = torch.zeros(M * k, N + c["pad"], dtype=_DTYPES[c["out"]], device=_dev())[:, :N]
        if E:
            chosen = _chosen(g, M, E, k, c["skew"]).reshape(-1)
            counts = torch.bincount(chosen, minlength=E)
            s["bounds"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
            s["splits"] = counts.tolist()       # rows of each group, known to who made the table
            # k == 1: rows that stand in the table's order already
            s["rows"] = torch.sort(chosen, stable=True).indices.int() if k > 1 else None
    elif c["op"] == "combine":
        T, d, k = c["T"], c["d"], c["k"]
        s["d"] = _rows(_normal(g, T * k, d), c["dtype"], c["pad"])
        s["weights"] = torch.softmax(_normal(g, T, k), -1)
        s["pos"] = torch.randperm(T * k, generator=g, device=_dev()).view(T, k).int()
        if c["idle"]:
            s["pos"][T - min(c["idle"], T):] = -1
        s["base"] = _rows(_normal(g, T, d), c["out"], c["pad"])
        s["y"] = _rows(torch.zeros(T, d, device=_dev()), c["out"], c["pad"])
    else:
        M, K, N, r, n = c["M"], c["K"], c["N"], c["r"], c["n"]
        s["x"] = _rows(_normal(g, M, K), c["dtype"], c["pad"])
        s["a"] = _weights(g, c["dtype"], n, r, K)
        s["b"] = _weights(g, c["dtype"], n, N, r)
        s["scales"] = 0.5 + torch.rand(n, generator=g, device=_dev())
        s["base"] = _rows(_normal(g, M, N), c["base"], c["pad"])
        s["out"] = _rows(torch.zeros(M, N, device=_dev()), c["out"], c["pad"])
        # runs of rows, one request each
        cuts = torch.sort(torch.randperm(M - 1, generator=g, device=_dev())[: c["runs"] - 1] + 1).values
        run = torch.zeros(M, dtype=torch.long, device=_dev())
        run[cuts] = 1
        ids = torch.randint(0, n, (c["runs"],), generator=g, device=_dev(), dtype=torch.int32)
        ids[torch.rand(c["runs"], generator=g, device=_dev()) < c["none"]] = -1
        s["adapters"] = ids[run.cumsum(0)].contiguous()
        if own:
            import moe_prefill_ffn_amd as mp

            s["workspace"] = torch.empty(mp.moe_lora_workspace_size(M, K, r), dtype=torch.uint8, device=_dev())
    return s


# ------------------------------------------------------------ plain forms ---

def _plain_group(s):
    c, E = s["case"], s["case"]["E"]
    e = s["eidx"].reshape(-1)
    order = torch.sort(torch.where(e < 0, E, e), stable=True)
    bounds = torch.searchsorted(order.values, torch.arange(E + 1, device=e.device, dtype=e.dtype)).int()
    place = torch.empty_like(e)
    place[order.indices] = torch.arange(e.numel(), device=e.device, dtype=torch.int32)
    inside = torch.arange(e.numel(), device=e.device) < bounds[E]
    rows = torch.where(inside, order.indices.int(), s["rows"])           # behind the last group: as they were
    return {"bounds": bounds, "rows": rows, "pos": torch.where(e < 0, -1, place).view(c["T"], c["k"])}


def _plain_product(s):
    c = s["case"]
    a = s["a"].float()
    if c["E"]:
        if s["rows"] is not None:
            a = a[(s["rows"] // c["k"]).long()]
        z = torch.cat([rows @ w.float().t() for rows, w in zip(a.split(s["splits"]), s["b"])])
    else:
        z = a @ s["b"][0].float().t()
    if c["swiglu"]:
        gate, up = z[:, : c["N"]], z[:, c["N"]:]
        z = gate / (1 + torch.exp(-gate)) * up
    return z.to(_DTYPES[c["out"]])


def _plain_combine(s):
    c = s["case"]
    pos, y = s["pos"], s["base"].float()
    for j in range(c["k"]):
        row = s["d"][pos[:, j].clamp(min=0).long()].float()
        y = y + torch.where(pos[:, j:j + 1] < 0, 0.0, s["weights"][:, j:j + 1] * row)
    return y.to(_DTYPES[c["out"]])


def _plain_lora(s):
    c = s["case"]
    x, y = s["x"].float(), s["base"].float().clone()      # the sum is not the base's: it is read again by the next pass
    for i in range(c["n"]):
        at = torch.nonzero(s["adapters"] == i).flatten()
        y[at] += (x[at] @ s["a"][i].float().t()) @ s["b"][i].float().t() * s["scales"][i]
    return y.to(_DTYPES[c["out"]])


# -------------------------------------------------------------------- run ---

def _own(s):
    import moe_prefill_ffn_amd as mp

    c = s["case"]
    if c["op"] == "group":
        mp.moe_group_rows(s["eidx"], c["E"], bounds=s["bounds"], rows=s["rows"], pos=s["pos"], workspace=s["workspace"])
        return {"bounds": s["bounds"], "rows": s["rows"], "pos": s["pos"]}
    if c["op"] == "product":
        if c["E"]:
            mp.moe_grouped_gemm(s["a"], s["b"], s["out"], bounds=s["bounds"], rows=s["rows"], top_k=c["k"], swiglu=c["swiglu"])
        else:
            mp.moe_grouped_gemm(s["a"], s["b"], s["out"], swiglu=c["swiglu"])
        return s["out"]
    if c["op"] == "combine":
        mp.moe_combine_rows(s["d"], s["weights"], s["pos"], s["y"], base=s["base"])
        return s["y"]
    mp.moe_lora_add(s["x"], s["a"], s["b"], s["adapters"], s["base"], s["out"], scales=s["scales"], workspace=s["workspace"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"group": _plain_group, "product": _plain_product, "combine": _plain_combine, "lora": _plain_lora}[state["case"]["op"]](state)


# ------------------------------------------------------------------- work ---

def _reached(n, draws):
    """How many of n are met by that many even draws, on average."""
    return n * (1 - (1 - 1 / n) ** draws)


def work(case):
    c = case
    if c["op"] == "group":
        pairs = c["T"] * c["k"]
        return {"bytes": 4.0 * (3 * pairs + c["E"] + 1), "flops": 1.0 * pairs}
    if c["op"] == "product":
        rows, wide = c["M"] * c["k"], c["N"] * (2 if c["swiglu"] else 1)
        groups = _reached(c["E"], rows) if c["E"] else 1
        if c["E"] and c["M"] == 1:
            groups = c["k"]
        return {"bytes": 2.0 * (c["M"] + groups * wide) * c["K"] + rows * c["N"] * _BYTES[c["out"]], "flops": 2.0 * rows * wide * c["K"]}
    if c["op"] == "combine":
        live = max(0, c["T"] - c["idle"])
        return {"bytes": 1.0 * c["d"] * (live * c["k"] * _BYTES[c["dtype"]] + 2 * c["T"] * _BYTES[c["out"]]) + 8.0 * c["T"] * c["k"],
                "flops": 2.0 * live * c["k"] * c["d"]}
    live = c["M"] * (1 - c["none"])
    used = _reached(c["n"], max(1.0, c["runs"] * (1 - c["none"])))
    return {"bytes": 2.0 * live * c["K"] + 2.0 * used * c["r"] * (c["K"] + c["N"]) + c["M"] * c["N"] * (_BYTES[c["base"]] + _BYTES[c["out"]]),
            "flops": 2.0 * live * c["r"] * (c["K"] + c["N"])}


# ------------------------------------------------------- 64-bit definition ---

def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "group":                      # one pair after the other, to the end of its expert's list
        lists = [[] for _ in range(c["E"])]
        pairs = s["eidx"].flatten().tolist()
        for p, e in enumerate(pairs):
            if e >= 0:
                lists[e].append(p)
        bounds, rows, pos = [0], [0] * len(pairs), [-1] * len(pairs)
        for members in lists:
            for at, p in enumerate(members, bounds[-1]):
                rows[at], pos[p] = p, at
            bounds.append(bounds[-1] + len(members))
        new = lambda v: torch.tensor(v, dtype=torch.int32, device=_dev())  # noqa: E731
        return {"bounds": new(bounds), "rows": new(rows), "pos": new(pos).view(c["T"], c["k"])}
    if c["op"] == "product":
        a, ends = s["a"].double(), s["bounds"].tolist() if c["E"] else [0, c["M"]]
        out = torch.empty(c["M"] * c["k"], c["N"], dtype=torch.float64, device=_dev())
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi == lo:
                continue
            part = a[lo:hi] if s.get("rows") is None else a[torch.div(s["rows"][lo:hi], c["k"], rounding_mode="floor").long()]
            z = torch.mm(part, s["b"][e].double().t())
            out[lo:hi] = z[:, : c["N"]] * torch.sigmoid(z[:, : c["N"]]) * z[:, c["N"]:] if c["swiglu"] else z
        return out
    if c["op"] == "combine":
        w = torch.where(s["pos"] < 0, 0.0, s["weights"].double())
        out = torch.empty(c["T"], c["d"], dtype=torch.float64, device=_dev())
        for lo in range(0, c["T"], 1024):       # a part of the tokens at a time
            t = slice(lo, lo + 1024)
            d = s["d"][s["pos"][t].clamp(min=0).long()].double()
            out[t] = s["base"][t].double() + (d * w[t, :, None]).sum(1)
        return out
    out = s["base"].double()
    for i in set(s["adapters"].tolist()) - {-1}:
        mask = s["adapters"] == i
        delta = (s["b"][i].double() @ (s["a"][i].double() @ s["x"][mask].double().t())).t()
        out[mask] = out[mask] + s["scales"][i].double() * delta
    return out
