"""Cases of the expert-layer operators: 8-bit products with block scales, the quantisers that make their
operands, routing, and combining the experts' rows.

`run` computes each operator in its plain form (elementary torch operations) or, with `own` set, by the
framework's entry points.  `exact` is the operator's definition in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "f32": torch.float32,
         "bf16": torch.bfloat16, "f16": torch.float16}
MAXIMA = {torch.float8_e4m3fn: 448.0, torch.float8_e5m2: 57344.0}


def _cdiv(a, b):
    return -(-a // b)


def listed():
    return [
        # A decode step's projection: 16 tokens against one large weight, bound by reading it.
        {"name": "product 16 tokens", "op": "product", "m": 16, "n": 14336, "k": 4096, "a": "e4m3",
         "b": "e4m3", "by": "tile", "out": "bf16"},
        # A gradient (e5m2) against a weight, every size odd, fp32 result.
        {"name": "product ragged", "op": "product", "m": 1023, "n": 1029, "k": 1000, "a": "e5m2",
         "b": "e4m3", "by": "tile", "out": "f32"},
        # A training-size linear layer.
        {"name": "product 8192", "op": "product", "m": 8192, "n": 8192, "k": 8192, "a": "e4m3",
         "b": "e4m3", "by": "tile", "out": "bf16"},
        # The experts' up projection in a prefill or training step: 4096 tokens times 8 choices.
        {"name": "product experts", "op": "experts", "m": 32768, "n": 2048, "k": 4096, "e": 64,
         "a": "e4m3", "b": "e4m3", "out": "bf16"},
        # The experts' weight gradients: each sums over its own tokens.
        {"name": "product depth", "op": "depth", "m": 2048, "n": 4096, "r": 16384, "e": 16,
         "a": "e5m2", "b": "e4m3", "out": "f32"},
        # Gathering and quantising the routed activations of a prefill or training step.
        {"name": "rows gathered", "op": "rows", "t": 4096, "c": 4096, "r": 32768, "in": "bf16",
         "q": "e4m3"},
        # Activations quantised along the tokens of each expert, for the weight gradient.
        {"name": "columns", "op": "columns", "r": 16384, "c": 4096, "e": 16, "in": "bf16",
         "q": "e4m3"},
        # Routing a decode batch: sigmoid scores, balancing bias, 4 of 8 groups.
        {"name": "route decode", "op": "route", "t": 64, "e": 256, "k": 8, "in": "f32",
         "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4, "renorm": True},
        # Routing a prefill or training batch: softmax scores.
        {"name": "route prefill", "op": "route", "t": 16384, "e": 128, "k": 8, "in": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renorm": True},
        # The router's gradient in training.
        {"name": "route backward", "op": "route_bwd", "t": 16384, "e": 256, "k": 8, "in": "f32",
         "score": "sigmoid", "renorm": True},
        # The experts' rows added up for each token.
        {"name": "combine", "op": "combine", "t": 4096, "k": 8, "c": 4096, "in": "bf16"},
        # Its gradient to the rows and to the routing weights.
        {"name": "combine backward", "op": "combine_bwd", "t": 8192, "k": 4, "c": 2048, "in": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm; one in three is a multiple of 16 where that fits."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.34:
        v -= v % 16
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["product", "product", "product", "experts", "experts", "depth", "rows", "tiles",
                     "columns", "route", "route", "route_bwd", "combine", "combine_bwd"])
    kind = lambda: rng.choice(["bf16", "bf16", "f16", "f32"])  # noqa: E731
    bits = lambda: rng.choice(["e4m3", "e4m3", "e5m2"])  # noqa: E731
    if op == "product":
        return {"op": op, "m": _log(rng, 1, 8192), "n": _log(rng, 64, 8192), "k": _log(rng, 64, 8192),
                "a": bits(), "b": "e4m3", "by": rng.choice(["tile", "tile", "row"]),
                "out": rng.choice(["bf16", "bf16", "f16", "f32"])}
    if op == "experts":
        e = _log(rng, 2, 128)
        n, k = _log(rng, 128, 4096), _log(rng, 128, 4096)
        while e * n * k > 64 * 2048 * 4096:
            n, k = max(128, n // 2), max(128, k // 2)
        return {"op": op, "m": _log(rng, 1, 16384), "n": n, "k": k, "e": e, "a": bits(), "b": "e4m3",
                "out": kind()}
    if op == "depth":
        return {"op": op, "m": _log(rng, 64, 2048), "n": _log(rng, 64, 2048), "r": _log(rng, 1, 16384),
                "e": _log(rng, 1, 32), "a": bits(), "b": "e4m3", "out": rng.choice(["f32", "bf16"])}
    if op == "rows":
        t = _log(rng, 1, 8192)
        return {"op": op, "t": t, "c": _log(rng, 64, 8192), "r": t * rng.choice([0, 1, 2, 4]),
                "in": kind(), "q": bits()}
    if op == "tiles":
        return {"op": op, "e": rng.choice([1, 1, 2, 5, 8]), "n": _log(rng, 64, 4096),
                "k": _log(rng, 64, 4096), "turn": rng.random() < 0.5, "in": kind(), "q": "e4m3"}
    if op == "columns":
        return {"op": op, "r": _log(rng, 1, 16384), "c": _log(rng, 64, 4096), "e": _log(rng, 1, 64),
                "in": kind(), "q": bits()}
    if op in ("route", "route_bwd"):
        e = rng.choice([8, 16, 60, 64, 96, 128, 160, 256, 384])
        g = rng.choice([1, 1, 2, 4])
        tg = rng.randint(1, g)
        k = rng.choice([1, 2, 4, 6, 8])
        k = min(k, e // g * tg)
        c = {"op": op, "t": _log(rng, 1, 16384), "e": e, "k": k, "in": kind(),
             "score": rng.choice(["softmax", "sigmoid"]), "renorm": rng.random() < 0.7}
        if op == "route_bwd" and k == 1:
            c["renorm"] = False  # one renormalised weight is 1: no gradient
        if op == "route":
            c |= {"bias": rng.random() < 0.5, "groups": g, "top_groups": tg}
        return c
    return {"op": op, "t": _log(rng, 1, 4096), "k": rng.choice([1, 2, 4, 6, 8]),
            "c": _log(rng, 64, 4096), "in": kind()}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, shape, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _activations(g, shape, dtype):
    """Rows of different sizes, a few outlying columns: what a layer's activations look like."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    x *= torch.exp(0.5 * torch.randn((shape[0], 1), generator=g, device="cuda"))
    x[:, ::97] *= 8.0
    return x.to(dtype)


def _operand(g, rows, cols, dtype, by):
    """An 8-bit matrix [rows, cols] whose rows start on 16-byte boundaries, and its scales."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    top, kb = MAXIMA[dtype], _cdiv(cols, BLOCK)
    store = torch.zeros((rows, _cdiv(cols, 16) * 16), dtype=dtype, device="cuda")
    q = store[:, :cols]
    q.copy_((x * (top / 5.0)).clamp_(-top, top))
    r = _cdiv(rows, BLOCK) if by == "tile" else rows
    s = torch.exp(0.5 * torch.randn((kb, r), generator=g, device="cuda")) * (5.0 / top)
    return q, (s.t().contiguous() if by == "tile" else s.t())


def _counts(g, rows, e):
    """How many of `rows` rows each of `e` experts gets: uneven, some without any."""
    p = torch.exp(0.7 * torch.randn(e, generator=g, device="cuda"))
    p[1::7] = 0.0
    c = torch.cumsum(p / p.sum(), 0)
    off = torch.round(c * rows).to(torch.int32)
    off[-1] = rows
    return torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), off])


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "product":
        s["a"], s["sa"] = _operand(g, case["m"], case["k"], TYPES[case["a"]], "row")
        s["b"], s["sb"] = _operand(g, case["n"], case["k"], TYPES[case["b"]], case["by"])
    elif op == "experts":
        e, n, k = case["e"], case["n"], case["k"]
        s["a"], s["sa"] = _operand(g, case["m"], k, TYPES[case["a"]], "row")
        b = torch.zeros((e, n, _cdiv(k, 16) * 16), dtype=TYPES[case["b"]], device="cuda")
        for i in range(e):
            b[i, :, :k] = (torch.randn((n, k), generator=g, device="cuda") * 89.6).clamp_(-448, 448).to(b.dtype)
        s["b"] = b[:, :, :k]
        s["sb"] = torch.exp(0.5 * torch.randn((e, _cdiv(n, BLOCK), _cdiv(k, BLOCK)), generator=g, device="cuda")) / 89.6
        s["offsets"] = _counts(g, case["m"], e)
        s["longest"] = int(s["offsets"].diff().max())
    elif op == "depth":
        e = case["e"]
        s["offsets"] = _counts(g, case["r"], e)
        width = (case["r"] // BLOCK + e) * BLOCK
        # Zeros follow the rows of an expert up to its next block.
        blocks = (s["offsets"].diff() + BLOCK - 1) // BLOCK
        first = torch.cumsum(blocks, 0) - blocks
        p = torch.arange(width, device="cuda")
        at = (torch.searchsorted(first * BLOCK, p, right=True) - 1).clamp(0, e - 1)
        full = (p - first[at] * BLOCK) < s["offsets"].diff()[at]
        for name, rows in (("a", case["m"]), ("b", case["n"])):
            q, s["s" + name] = _operand(g, rows, width, TYPES[case[name]], "row")
            s[name] = torch.where(full, q.float(), 0.0).to(q.dtype)
        s["longest"] = int(blocks.max()) * BLOCK
    elif op == "rows":
        s["x"] = _activations(g, (case["t"], case["c"]), TYPES[case["in"]])
        s["rows"] = (torch.randint(0, case["t"], (case["r"],), generator=g, device="cuda", dtype=torch.int32)
                     if case["r"] else None)
    elif op == "tiles":
        s["x"] = 0.02 * _randn(g, (case["e"], case["n"], case["k"]))
        s["x"] = s["x"].to(TYPES[case["in"]])
    elif op == "columns":
        s["x"] = _activations(g, (case["r"], case["c"]), TYPES[case["in"]])
        s["offsets"] = _counts(g, case["r"], case["e"])
    elif op in ("route", "route_bwd"):
        t, e = case["t"], case["e"]
        s["logits"] = (1.5 * _randn(g, (t, e))).to(TYPES[case["in"]])
        s["bias"] = 0.1 * _randn(g, (e,)) if case.get("bias") else None
        if op == "route_bwd":
            s["ids"] = torch.argsort(s["logits"].float(), dim=1, descending=True, stable=True)[:, :case["k"]].to(torch.int32).contiguous()
            s["dw"] = _randn(g, (t, case["k"]))
    else:
        t, k, c, kind = case["t"], case["k"], case["c"], TYPES[case["in"]]
        s["x"] = _randn(g, (t * k, c), kind)
        s["slots"] = torch.randperm(t * k, generator=g, device="cuda").to(torch.int32).reshape(t, k)
        w = torch.rand((t, k), generator=g, device="cuda") + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        if op == "combine_bwd":
            s["dy"] = _randn(g, (t, c), kind)
    return s


# ---------------------------------------------------------------- plain forms

def _spread(s, rows, cols, by):
    """Scales of blocks of 128, one for each element."""
    s = s.repeat_interleave(BLOCK, dim=-1)[..., :cols]
    return s.repeat_interleave(BLOCK, dim=-2)[..., :rows, :] if by == "tile" else s


def _values(q, s, by):
    return q.float() * _spread(s, q.shape[-2], q.shape[-1], by)


def _positions(first, count, longest):
    """[e, longest] places first[e] + i, and which of them are among the `count[e]`."""
    i = torch.arange(longest, device=first.device)
    return first[:, None] + i, i < count[:, None]


def _quantise(x, dtype, dims):
    """Blocks of x (their values along `dims`) in 8 bits, and the scales."""
    amax = x.abs().amax(dim=dims, keepdim=True).clamp(min=MAXIMA[dtype] * 2.0 ** -126)
    top = torch.full_like(amax, MAXIMA[dtype])  # a number here would be multiplied by a rounded reciprocal
    return (x * (top / amax)).to(dtype), amax / top


def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[-1], 0, rows - x.shape[-2]))


def _plain_route(s, case):
    l = s["logits"].double()
    t, e = l.shape
    k = case["k"]
    if case["score"] == "softmax":
        m = l.amax(1, keepdim=True)
        x = torch.exp(l - torch.where(m == -math.inf, 0.0, m))
        z = x.sum(1, keepdim=True)
        p = torch.where(z == 0, 0.0, x / z)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    b = p if s["bias"] is None else p + s["bias"].double()
    b = torch.where(torch.isnan(b), -math.inf, b)
    g = case["groups"]
    if case["top_groups"] < g:
        best = b.reshape(t, g, e // g).topk(min(2, e // g), dim=2).values.sum(2)
        rank = torch.sort(best, dim=1, descending=True, stable=True).indices
        keep = torch.zeros((t, g), dtype=torch.bool, device=l.device)
        keep.scatter_(1, rank[:, :case["top_groups"]], True)
        b = torch.where(keep.repeat_interleave(e // g, dim=1), b, -math.inf)
    ids = torch.sort(b, dim=1, descending=True, stable=True).indices[:, :k]
    w = p.gather(1, ids)
    if case["renorm"]:
        z = w.sum(1, keepdim=True)
        w = torch.where(z == 0, 0.0, w / z)
    flat, order = torch.sort(ids.reshape(-1), stable=True)
    offsets = torch.searchsorted(flat, torch.arange(e + 1, device=l.device))
    slots = torch.empty_like(order)
    slots[order] = torch.arange(t * k, device=l.device)
    i32 = torch.int32
    return {"weights": w.float(), "ids": ids.to(i32), "offsets": offsets.to(i32),
            "tokens": (order // k).to(i32), "slots": slots.reshape(t, k).to(i32)}


def _route_gradient(s, case, kind):
    """The gradient to the logits, in numbers of type `kind`."""
    l, ids, dw = s["logits"].to(kind), s["ids"].long(), s["dw"].to(kind)
    p = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
    w = p.gather(1, ids)
    if case["renorm"]:
        z = w.sum(1, keepdim=True)
        dw = (dw - (dw * w / z).sum(1, keepdim=True)) / z
    dp = torch.zeros_like(p).scatter_(1, ids, dw)
    if case["score"] == "softmax":
        return p * (dp - (dp * p).sum(1, keepdim=True))
    return dp * p * (1 - p)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "product":
        return (_values(s["a"], s["sa"], "row") @ _values(s["b"], s["sb"], case["by"]).t()).to(TYPES[case["out"]])
    if op == "experts":
        a, b = _values(s["a"], s["sa"], "row"), _values(s["b"], s["sb"], "tile")
        at, there = _positions(s["offsets"][:-1], s["offsets"].diff(), s["longest"])
        each = torch.bmm(a[at.clamp(max=len(a) - 1)], b.transpose(1, 2))
        e = torch.searchsorted(s["offsets"][1:], torch.arange(len(a), device=a.device), right=True)
        return each[e, torch.arange(len(a), device=a.device) - s["offsets"][e]].to(TYPES[case["out"]])
    if op == "depth":
        a, b = _values(s["a"], s["sa"], "row"), _values(s["b"], s["sb"], "row")
        blocks = (s["offsets"].diff() + BLOCK - 1) // BLOCK
        at, there = _positions((torch.cumsum(blocks, 0) - blocks) * BLOCK, blocks * BLOCK, s["longest"])
        at = at.clamp(max=a.shape[1] - 1)
        each = torch.where(there, a[:, at], 0.0).transpose(0, 1)
        return torch.bmm(each, b[:, at].permute(1, 2, 0)).to(TYPES[case["out"]])
    if op == "rows":
        x = s["x"] if s["rows"] is None else s["x"][s["rows"]]
        r, c = x.shape
        kb = _cdiv(c, BLOCK)
        q, sc = _quantise(_pad(x.float(), r, kb * BLOCK).reshape(r, kb, BLOCK), TYPES[case["q"]], 2)
        return q.reshape(r, kb * BLOCK)[:, :c], sc.reshape(r, kb)
    if op == "tiles":
        x = s["x"].float()
        e, n, k = x.shape
        nb, kb = _cdiv(n, BLOCK), _cdiv(k, BLOCK)
        q, sc = _quantise(_pad(x, nb * BLOCK, kb * BLOCK).reshape(e, nb, BLOCK, kb, BLOCK), TYPES[case["q"]], (2, 4))
        q, sc = q.reshape(e, nb * BLOCK, kb * BLOCK)[:, :n, :k], sc.reshape(e, nb, kb)
        return (q.transpose(1, 2), sc.transpose(1, 2)) if case["turn"] else (q, sc)
    if op == "columns":
        x, off = s["x"].float(), s["offsets"]
        r, c = x.shape
        width = r // BLOCK + case["e"]
        blocks = (off.diff() + BLOCK - 1) // BLOCK
        first = torch.cumsum(blocks, 0) - blocks
        e = torch.searchsorted(off[1:], torch.arange(r, device=x.device), right=True)
        to = first[e] * BLOCK + torch.arange(r, device=x.device) - off[e]
        y = torch.zeros((width * BLOCK, c), device=x.device).index_copy_(0, to, x)
        q, sc = _quantise(y.reshape(width, BLOCK, c), TYPES[case["q"]], 1)
        return q.reshape(width * BLOCK, c).t(), sc.reshape(width, c).t()
    if op == "route":
        return _plain_route(s, case)
    if op == "route_bwd":
        return _route_gradient(s, case, torch.float32).to(s["logits"].dtype)
    x, slots, w = s["x"], s["slots"], s["w"]
    if op == "combine":
        return (x[slots].float() * w[:, :, None]).sum(1).to(x.dtype)
    dy = s["dy"].float()
    dx = torch.empty_like(x)
    dx[slots] = (dy[:, None, :] * w[:, :, None]).to(x.dtype)
    return dx, (x[slots].float() * dy[:, None, :]).sum(2)


# ---------------------------------------------------------------- the framework's

def _own(s):
    import dense_gemm_05_gb300 as dg
    case = s["case"]
    op = case["op"]
    if op == "product":
        return dg.matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], out_dtype=TYPES[case["out"]])
    if op == "experts":
        return dg.matmul_fp8(s["a"], s["sa"], s["b"], s["sb"], offsets=s["offsets"], out_dtype=TYPES[case["out"]])
    if op == "depth":
        return dg.matmul_fp8_depth(s["a"], s["sa"], s["b"], s["sb"], s["offsets"], out_dtype=TYPES[case["out"]])
    if op == "rows":
        return dg.quantize_fp8_rows(s["x"], rows=s["rows"], dtype=TYPES[case["q"]])
    if op == "tiles":
        return dg.quantize_fp8_tiles(s["x"], transpose=case["turn"], dtype=TYPES[case["q"]])
    if op == "columns":
        return dg.quantize_fp8_columns(s["x"], offsets=s["offsets"], dtype=TYPES[case["q"]])
    if op == "route":
        return dg.route(s["logits"], case["k"], score=case["score"], bias=s["bias"], groups=case["groups"],
                        top_groups=case["top_groups"], renormalize=case["renorm"])._asdict()
    if op == "route_bwd":
        return dg.route_backward(s["dw"], s["logits"], s["ids"], score=case["score"], renormalize=case["renorm"])
    if op == "combine":
        return dg.combine(s["x"], s["slots"], s["w"])
    return dg.combine_backward(s["dy"], s["x"], s["slots"], s["w"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_values(q, s, by):
    v = q.double()
    for b in range(_cdiv(v.shape[-1], BLOCK)):
        cols = slice(b * BLOCK, (b + 1) * BLOCK)
        if by == "row":
            v[..., cols] *= s[..., b:b + 1].double()
        else:
            for r in range(_cdiv(v.shape[-2], BLOCK)):
                v[..., r * BLOCK:(r + 1) * BLOCK, cols] *= s[..., r:r + 1, b:b + 1].double()
    return v


def _round8(v, dtype):
    """The nearest values of an 8-bit type (ties to even) of numbers within its range."""
    mantissa, low = (3, -6) if dtype == torch.float8_e4m3fn else (2, -14)
    e = torch.frexp(v).exponent - 1
    step = torch.ldexp(torch.ones_like(v), e.clamp(min=low) - mantissa)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        return _exact_values(s["a"], s["sa"], "row") @ _exact_values(s["b"], s["sb"], case["by"]).t()
    if op == "experts":
        if 2 * case["m"] * case["n"] * case["k"] > 1e13:
            return None
        a = _exact_values(s["a"], s["sa"], "row")
        out, off = [], s["offsets"].tolist()
        for e in range(case["e"]):
            if off[e + 1] > off[e]:
                out.append(a[off[e]:off[e + 1]] @ _exact_values(s["b"][e], s["sb"][e], "tile").t())
        return torch.cat(out)
    if op == "depth":
        a, b = _exact_values(s["a"], s["sa"], "row"), _exact_values(s["b"], s["sb"], "row")
        out, at, off = [], 0, s["offsets"].tolist()
        for e in range(case["e"]):
            w = _cdiv(off[e + 1] - off[e], BLOCK) * BLOCK
            out.append(a[:, at:at + w] @ b[:, at:at + w].t())
            at += w
        return torch.stack(out)
    if op in ("rows", "tiles", "columns"):
        dtype = TYPES[case["q"]]
        top = MAXIMA[dtype]
        x = s["x"].double()
        if op == "rows":
            x = x if s["rows"] is None else x[s["rows"].long()]
            q, sc = torch.empty_like(x), []
            for b in range(0, x.shape[1], BLOCK):
                sc.append(x[:, b:b + BLOCK].abs().amax(1).clamp(min=top * 2.0 ** -126) / top)
                q[:, b:b + BLOCK] = _round8(x[:, b:b + BLOCK] / sc[-1][:, None], dtype)
            return q, torch.stack(sc, 1)
        if op == "columns":
            off, width = s["offsets"].tolist(), x.shape[0] // BLOCK + case["e"]
            q = torch.zeros((x.shape[1], width * BLOCK), dtype=torch.float64, device=x.device)
            sc = torch.full((x.shape[1], width), 2.0 ** -126, dtype=torch.float64, device=x.device)
            at = 0
            for e in range(case["e"]):
                for i in range(off[e], off[e + 1], BLOCK):
                    y = x[i:min(i + BLOCK, off[e + 1])].t()
                    sc[:, at] = y.abs().amax(1).clamp(min=top * 2.0 ** -126) / top
                    q[:, at * BLOCK:at * BLOCK + y.shape[1]] = _round8(y / sc[:, at:at + 1], dtype)
                    at += 1
            return q, sc
        n, k = x.shape[1:]
        q = torch.empty_like(x)
        sc = torch.empty((x.shape[0], _cdiv(n, BLOCK), _cdiv(k, BLOCK)), dtype=torch.float64, device=x.device)
        for i in range(sc.shape[1]):
            for j in range(sc.shape[2]):
                at = (slice(None), slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
                sc[:, i, j] = x[at].abs().amax((1, 2)).clamp(min=top * 2.0 ** -126) / top
                q[at] = _round8(x[at] / sc[:, i, j][:, None, None], dtype)
        return (q.transpose(1, 2), sc.transpose(1, 2)) if case["turn"] else (q, sc)
    if op == "route":
        p = s["logits"].double()
        p = torch.softmax(p, 1) if case["score"] == "softmax" else torch.sigmoid(p)
        b = p if s["bias"] is None else p + s["bias"].double()
        t, e = p.shape
        g = case["groups"]
        if case["top_groups"] < g:
            best = b.view(t, g, -1).sort(2, descending=True).values[:, :, :2].sum(2)
            # a group is kept if fewer than top_groups are better, or as good and before it
            ahead = (best[:, None, :] > best[:, :, None]) | ((best[:, None, :] == best[:, :, None]) & (
                torch.arange(g, device=p.device)[None, :] < torch.arange(g, device=p.device)[:, None]))
            b = b.masked_fill((ahead.sum(2) >= case["top_groups"]).repeat_interleave(e // g, 1), -math.inf)
        w = []
        for _ in range(case["k"]):
            best = b.amax(1, keepdim=True)
            first = (b == best).int().argmax(1, keepdim=True)
            w.append(p.gather(1, first))
            b = b.scatter(1, first, -math.inf)
        w = torch.cat(w, 1)
        return {"weights": w / w.sum(1, keepdim=True) if case["renorm"] else w, "ids": None, "offsets": None,
                "tokens": None, "slots": None}
    if op == "route_bwd":
        l = s["logits"].double().requires_grad_()
        p = torch.softmax(l, 1) if case["score"] == "softmax" else torch.sigmoid(l)
        w = p.gather(1, s["ids"].long())
        w = w / w.sum(1, keepdim=True) if case["renorm"] else w
        (w * s["dw"].double()).sum().backward()
        return l.grad
    x, slots, w = s["x"].double(), s["slots"].long(), s["w"].double()
    if op == "combine":
        y = torch.zeros((case["t"], case["c"]), dtype=torch.float64, device=x.device)
        for j in range(case["k"]):
            y += w[:, j:j + 1] * x[slots[:, j]]
        return y
    dy, dx, dw = s["dy"].double(), torch.empty_like(x), torch.empty_like(w)
    for j in range(case["k"]):
        dx[slots[:, j]] = w[:, j:j + 1] * dy
        dw[:, j] = (x[slots[:, j]] * dy).sum(1)
    return dx, dw


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1, "e5m2": 1}
    if op in ("product", "experts"):
        m, n, k = case["m"], case["n"], case["k"]
        kb, e = _cdiv(k, BLOCK), min(case.get("e", 1), m)
        sb = n if case.get("by") == "row" else _cdiv(n, BLOCK)
        return {"bytes": m * k + 4 * m * kb + e * (n * k + 4 * sb * kb) + m * n * size[case["out"]],
                "flops": 2 * m * n * k}
    if op == "depth":
        m, n, r, e = case["m"], case["n"], case["r"], case["e"]
        return {"bytes": (m + n) * (r + 4 * _cdiv(r, BLOCK)) + e * m * n * size[case["out"]],
                "flops": 2 * m * n * r}
    if op == "rows":
        r, c = case["r"] or case["t"], case["c"]
        return {"bytes": min(r, case["t"]) * c * size[case["in"]] + r * (c + 4 * _cdiv(c, BLOCK)) + 4 * case["r"],
                "flops": 3 * r * c}
    if op == "tiles":
        e, n, k = case["e"], case["n"], case["k"]
        return {"bytes": e * (n * k * (size[case["in"]] + 1) + 4 * _cdiv(n, BLOCK) * _cdiv(k, BLOCK)),
                "flops": 3 * e * n * k}
    if op == "columns":
        r, c, width = case["r"], case["c"], case["r"] // BLOCK + case["e"]
        return {"bytes": r * c * size[case["in"]] + width * (BLOCK + 4) * c, "flops": 3 * r * c}
    if op in ("route", "route_bwd"):
        t, e, k, b = case["t"], case["e"], case["k"], size[case["in"]]
        if op == "route":
            return {"bytes": t * e * b + 16 * t * k + 4 * (e + 1) + 4 * e * bool(case["bias"]), "flops": 8 * t * e}
        return {"bytes": 2 * t * e * b + 8 * t * k, "flops": 8 * t * e}
    t, k, c, b = case["t"], case["k"], case["c"], size[case["in"]]
    if op == "combine":
        return {"bytes": t * k * c * b + t * c * b + 8 * t * k, "flops": 2 * t * k * c}
    return {"bytes": 2 * t * k * c * b + t * c * b + 12 * t * k, "flops": 3 * t * k * c}
