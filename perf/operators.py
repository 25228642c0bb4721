"""Cases, plain forms and exact values of the mixture-of-experts and 8-bit operators.

A training step of a dense or expert layer around the Muon step: routing of tokens to
experts, quantisation to 8 bits with a power-of-two scale for each block of 128, the
products in that form (forward, input gradient and weight gradient are the same product
of differently laid out operands), the experts' products over ragged groups of rows, and
the weighted sum of the experts' outputs. `own` chooses between the plain form below and
this repository's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FMT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP_EXPONENT = {"e4m3": 8, "e5m2": 15}     # the largest value is 1.75 * 2^this in both formats
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ----------------------------------------------------------------------------- cases

def listed():
    """Sizes: a 7B-class layer (4096, 11008), a smaller one (2048, 5632) and a batch of 64
    experts (1408 x 2048), as this repository's workloads have them."""
    return [
        # one decoding step of 16 sequences: latency alone
        {"name": "route decode", "op": "route", "tokens": 16, "experts": 64, "top_k": 6, "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "type": "bf16", "align": 16},
        # a training batch through a router with a balance bias and expert groups
        {"name": "route batch", "op": "route", "tokens": 16384, "experts": 64, "top_k": 6, "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "type": "f32", "align": 128},
        # its gradient, dense through the softmax
        {"name": "route gradient", "op": "route_gradient", "tokens": 16384, "experts": 64, "top_k": 6,
         "score": "softmax", "type": "f32"},
        # activations of a dense layer: rows for the forward product, columns for the weight gradient
        {"name": "quantize activations", "op": "quantize", "batch": 1, "rows": 8192, "cols": 4096, "type": "bf16",
         "format": "e4m3", "blocks": False, "gather": 0},
        # one kind of expert weights out of the fp32 masters, once a step, both orientations
        {"name": "quantize expert weights", "op": "quantize", "batch": 64, "rows": 1408, "cols": 2048, "type": "f32",
         "format": "e4m3", "blocks": True, "gather": 0},
        # one token through a projection: the weights are read once
        {"name": "product one token", "op": "product", "m": 1, "n": 11008, "k": 4096, "type": "bf16",
         "formats": "e4m3 e4m3"},
        # the forward product of a large batch
        {"name": "product forward", "op": "product", "m": 8192, "n": 11008, "k": 4096, "type": "bf16",
         "formats": "e4m3 e4m3"},
        # a weight gradient in fp32 over an odd number of tokens, output gradients with the wider range
        {"name": "product weight gradient", "op": "product", "m": 5632, "n": 2048, "k": 16383, "type": "f32",
         "formats": "e5m2 e4m3"},
        # one projection of all experts over a routed batch: 64 ragged groups of rows
        {"name": "experts forward", "op": "experts", "tokens": 8192, "experts": 64, "top_k": 6, "n": 1408, "k": 2048,
         "type": "bf16", "formats": "e4m3 e4m3"},
        # the same experts' weight gradients: 64 ragged contractions
        {"name": "experts weight gradient", "op": "experts_gradient", "tokens": 8192, "experts": 64, "top_k": 6,
         "n": 1408, "k": 2048, "type": "bf16", "formats": "e5m2 e4m3"},
        # each token's weighted sum of its experts' rows, and its gradient
        {"name": "combine", "op": "combine", "tokens": 8192, "experts": 64, "top_k": 6, "cols": 2048, "type": "bf16"},
        {"name": "combine gradient", "op": "combine_gradient", "tokens": 8192, "experts": 64, "top_k": 6,
         "cols": 2048, "type": "bf16"},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["route", "route_gradient", "quantize", "product", "product", "experts", "experts_gradient",
                     "combine", "combine_gradient"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("route", "route_gradient"):
        experts = rng.choice([8, 16, 40, 64, 96, 128, 160, 256])
        c = {"op": op, "tokens": _spread(rng, 1, 16384), "experts": experts, "top_k": rng.randint(1, 8),
             "score": rng.choice(["softmax", "sigmoid"]), "type": kind}
        if op == "route":
            groups = rng.choice([1, 1, 4, 8])
            c.update(bias=rng.random() < 0.5, groups=groups, top_groups=max(1, groups // 2),
                     align=rng.choice([1, 16, 128]))
            c["top_k"] = min(c["top_k"], experts // groups * c["top_groups"])
        return c
    if op == "quantize":
        blocks = rng.random() < 0.4
        batch = rng.choice([1, 1, 8]) if blocks else 1
        rows = _spread(rng, 1, 16384)
        cols = _spread(rng, 1, min(11008, max(1, (1 << 26) // (rows * batch))))
        return {"op": op, "batch": batch, "rows": rows, "cols": cols, "type": kind,
                "format": rng.choice(["e4m3", "e5m2"]), "blocks": blocks,
                "gather": 0 if blocks else rng.choice([0, 0, 1, 6])}
    formats = rng.choice(["e4m3 e4m3", "e4m3 e4m3", "e5m2 e4m3", "e4m3 e5m2", "e5m2 e5m2"])
    if op == "product":
        return {"op": op, "m": rng.choice([1, _spread(rng, 1, 64), _spread(rng, 1, 8192)]),
                "n": _spread(rng, 16, 11008), "k": _spread(rng, 16, 4096), "type": kind, "formats": formats}
    c = {"op": op, "tokens": _spread(rng, 1, 8192), "experts": rng.choice([8, 16, 40, 64]), "top_k": rng.randint(1, 6),
         "type": kind}
    if op in ("combine", "combine_gradient"):
        c["cols"] = _spread(rng, 16, 2048)
    else:
        c.update(n=_spread(rng, 16, 1408), k=_spread(rng, 16, 2048), formats=formats)
    return c


# ----------------------------------------------------------------------------- inputs

def _up(n, to):
    return (n + to - 1) // to * to


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activations(g, rows, cols):
    """Normal values with a few loud channels, as layer inputs have them."""
    return _normal(g, rows, cols) * torch.exp(0.7 * _normal(g, cols))


def _logits(g, c):
    """Router logits with popular and unpopular experts."""
    return (1.5 * _normal(g, c["tokens"], c["experts"]) + 0.5 * _normal(g, c["experts"])).to(TYPES[c["type"]])


def _chosen(g, c):
    """Distinct experts of each token, popular ones more often."""
    noise = _normal(g, c["tokens"], c["experts"]) + 0.5 * _normal(g, c["experts"])
    return noise.topk(c["top_k"], dim=1).indices.to(torch.int32)


def _capacity(slots, experts, align):
    """Rows that any routing of `slots` rows to the experts can need."""
    return slots + experts * (align - 1)


def _order(ids, experts, align):
    """Stable order of the flat slots by expert, each expert's rows padded to `align`."""
    flat = ids.reshape(-1).to(torch.int64)
    counts = (flat[:, None] == torch.arange(experts, device=flat.device)).sum(0)
    ends = ((counts + align - 1) // align * align).cumsum(0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends])
    slots = torch.argsort(flat, stable=True)
    slots = slots[flat[slots] >= 0]
    first = torch.cat([torch.zeros_like(ends[:1]), counts.cumsum(0)])
    expert = flat[slots]
    to = offsets[expert] + torch.arange(len(slots), device=flat.device) - first[expert]
    rows = torch.full((_capacity(len(flat), experts, align),), -1, dtype=torch.int32, device=flat.device)
    rows[to] = slots.to(torch.int32)
    pos = torch.full((len(flat),), -1, dtype=torch.int32, device=flat.device)
    pos[slots] = to.to(torch.int32)
    return offsets.to(torch.int32), counts.to(torch.int32), rows, pos.view(ids.shape)


def _operand(g, rows, cols, fmt, weights=False):
    """A quantised operand [rows, cols] whose scales run along its rows."""
    x = 0.02 * _normal(g, rows, cols) if weights else _activations(g, rows, cols)
    return _quantize_rows(x, fmt)


def _routed(g, c, cols, fmt, by_column):
    """Rows of routed tokens in expert order, padding rows zero, quantised along the rows or,
    for the weight gradients, along each column (the transposed operand)."""
    x = _activations(g, c["tokens"], cols)
    rows = c["rows_of"]
    x = torch.where(rows[:, None] >= 0, x[rows.clamp(min=0).long() // c["top_k"]], 0.0)
    return _quantize_rows(x.t().contiguous() if by_column else x, fmt)


def prepare(case, seed):
    g, c = _generator(seed), dict(case)
    op = c["op"]
    if op in ("route", "route_gradient"):
        c["logits"] = _logits(g, c)
        c["bias_values"] = 0.1 * _normal(g, c["experts"]) if c.get("bias") else None
        if op == "route_gradient":
            c["ids"] = c["logits"].float().topk(c["top_k"], dim=1).indices.to(torch.int32)
            c["dweights"] = _normal(g, c["tokens"], c["top_k"])
    elif op == "quantize":
        source = -(-c["rows"] // max(1, c["gather"]))
        x = torch.stack([_activations(g, source, c["cols"]) for _ in range(c["batch"])])
        c["x"] = x.to(TYPES[c["type"]])
        if c["gather"]:   # the rows of a routed batch: tokens in another order, some rows padding
            index = torch.randperm(c["rows"], generator=g, device=DEV).to(torch.int32)
            pad = torch.rand(c["rows"], generator=g, device=DEV) < 0.05
            c["index"] = torch.where(pad, -1, index)
    elif op == "product":
        fa, fb = c["formats"].split()
        c["a"] = _operand(g, c["m"], c["k"], fa)
        c["b"] = _operand(g, c["n"], c["k"], fb, weights=True)
    else:
        ids = _chosen(g, c)
        c["offsets"], counts, c["rows_of"], c["pos"] = _order(ids, c["experts"], 128)
        c["most"] = _up(int(counts.max()), 128)
        cap = _up(len(c["rows_of"]), 128)
        c["rows_of"] = torch.nn.functional.pad(c["rows_of"], (0, cap - len(c["rows_of"])), value=-1)
        if op in ("combine", "combine_gradient"):
            c["o"] = (0.5 * _normal(g, cap, c["cols"])).to(TYPES[c["type"]])
            c["weights"] = torch.softmax(_normal(g, c["tokens"], c["top_k"]), 1)
            if op == "combine_gradient":
                c["dy"] = _normal(g, c["tokens"], c["cols"]).to(TYPES[c["type"]])
                c["do"] = torch.zeros_like(c["o"])
        else:
            fa, fb = c["formats"].split()
            if op == "experts":
                c["a"] = _routed(g, c, c["k"], fa, False)
                q, s = _operand(g, c["experts"] * c["n"], c["k"], fb, weights=True)
                c["b"] = (q.view(c["experts"], c["n"], -1), s.view(c["experts"], c["n"], -1))
                c["out"] = torch.zeros(cap, c["n"], dtype=TYPES[c["type"]], device=DEV)
            else:
                c["a"] = _routed(g, c, c["n"], fa, True)
                c["b"] = _routed(g, c, c["k"], fb, True)
    return c


# ----------------------------------------------------------------------------- plain forms

def _power(e):
    """2^e as float32, e in [-126, 127], from its bits."""
    return ((e + 127) << 23).view(torch.float32)


def _to_scale(e):
    """Scale bytes 2^e, padded with ones to a multiple of four blocks."""
    e = torch.nn.functional.pad(e, (0, -e.shape[-1] % 4))
    return (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _scale_of(amax, fmt):
    """The least e with amax <= 1.75 * 2^(top + e); 0 for a block of zeros."""
    half, ex = torch.frexp(amax)
    e = ex - 1 - TOP_EXPONENT[fmt] + (half > 0.875).to(torch.int32)
    return torch.where(amax > 0, e.clamp(min=-126), 0).to(torch.int32)


def _quantize_rows(x, fmt):
    """[..., rows, cols] -> values padded to 128 columns, one scale per 128 of a row."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % 128))
    b = x.unflatten(-1, (-1, 128))
    e = _scale_of(b.abs().amax(-1), fmt)
    return (b * _power(-e)[..., None]).flatten(-2).to(FMT[fmt]), _to_scale(e)


def _quantize_blocks(x, fmt):
    """As _quantize_rows with one scale per 128 x 128, kept for each row."""
    rows = x.shape[-2]
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[-1] % 128, 0, -rows % 128))
    b = x.unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    e = _scale_of(b.abs().amax((-3, -1)), fmt)
    q = (b * _power(-e)[..., :, None, :, None]).flatten(-2).flatten(-3, -2)[..., :rows, :].to(FMT[fmt])
    return q, _to_scale(e.repeat_interleave(128, -2)[..., :rows, :])


def _values(operand, cols=None):
    q, s = operand
    blocks = q.shape[-1] // 128
    return (q.float().unflatten(-1, (blocks, 128)) * s.float()[..., :blocks, None]).flatten(-2)


def _run_quantize(c):
    x = c["x"]
    if c["gather"]:
        i = c["index"]
        x = torch.where(i[:, None] >= 0, x[0][i.clamp(min=0).long() // c["gather"]], 0.0)[None]
    f = _quantize_blocks if c["blocks"] else _quantize_rows
    return f(x, c["format"]) + f(x.transpose(-1, -2).contiguous(), c["format"])


def _scores(logits, score):
    l = logits.double()
    return torch.softmax(l, 1) if score == "softmax" else 1.0 / (1.0 + torch.exp(-l))


def _run_route(c):
    s = _scores(c["logits"], c["score"])
    key = s if c["bias_values"] is None else s + c["bias_values"].double()
    if c["groups"] > 1:
        of = key.unflatten(1, (c["groups"], -1))
        best = of.sort(dim=2, descending=True, stable=True).values[:, :, :2].sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        mask = torch.zeros_like(best, dtype=torch.bool).scatter(1, kept, True)
        key = torch.where(mask[:, :, None], of, -math.inf).flatten(1)
    ids = key.sort(dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    w = s.gather(1, ids)
    w = w / (w.sum(1, keepdim=True) + 1e-20)
    offsets, counts, rows, pos = _order(ids.to(torch.int32), c["experts"], c["align"])
    return ids.to(torch.int32), w.float(), offsets, counts, rows, pos


def _run_route_gradient(c):
    s = _scores(c["logits"], c["score"])
    ids = c["ids"].long()
    chosen = s.gather(1, ids)
    total = chosen.sum(1, keepdim=True) + 1e-20
    dw = c["dweights"].double()
    ds = (dw - (dw * chosen / total).sum(1, keepdim=True)) / total
    if c["score"] == "sigmoid":
        d = torch.zeros_like(s).scatter(1, ids, ds * chosen * (1.0 - chosen))
    else:
        d = s * (torch.zeros_like(s).scatter(1, ids, ds) - (ds * chosen).sum(1, keepdim=True))
    return d.to(c["logits"].dtype)


def _run_product(c):
    return (_values(c["a"]) @ _values(c["b"]).t()).to(TYPES[c["type"]])


def _spans(c):
    """Row numbers of each expert, [experts, most], and which of them it has."""
    at = c["offsets"][:-1, None].long() + torch.arange(c["most"], device=DEV)
    return at.clamp(max=len(c["rows_of"]) - 1), at < c["offsets"][1:, None]


def _run_experts(c):
    at, has = _spans(c)
    a = _values(c["a"])[at]
    y = torch.bmm(a, _values(c["b"]).transpose(1, 2).contiguous())
    c["out"][at[has]] = y[has].to(c["out"].dtype)
    return c["out"]


def _run_experts_gradient(c):
    at, has = _spans(c)
    a = (_values(c["a"])[:, at] * has).transpose(0, 1).contiguous()
    b = (_values(c["b"])[:, at] * has).permute(1, 2, 0).contiguous()
    return torch.bmm(a, b).to(TYPES[c["type"]])


def _run_combine(c):
    picked = c["o"].float()[c["pos"].long()]
    return (picked * c["weights"][:, :, None]).sum(1).to(c["o"].dtype)


def _run_combine_gradient(c):
    at = c["pos"].long()
    dy = c["dy"].float()
    dw = (c["o"].float()[at] * dy[:, None, :]).sum(2)
    c["do"][at] = (c["weights"][:, :, None] * dy[:, None, :]).to(c["do"].dtype)
    return dw, c["do"]


PLAIN = {"route": _run_route, "route_gradient": _run_route_gradient, "quantize": _run_quantize,
         "product": _run_product, "experts": _run_experts, "experts_gradient": _run_experts_gradient,
         "combine": _run_combine, "combine_gradient": _run_combine_gradient}


# ----------------------------------------------------------------------------- this repository's calls

def _run_own(c):
    import newton_schulz_step_amd as nss
    op = c["op"]
    if op == "route":
        h = nss.route_hyper(score=c["score"], top_k=c["top_k"], n_groups=c["groups"], top_groups=c["top_groups"])
        ids, w = nss.route(c["logits"], h, bias=c["bias_values"])
        return (ids, w) + tuple(nss.expert_order(ids, c["experts"], align=c["align"]))
    if op == "route_gradient":
        h = nss.route_hyper(score=c["score"], top_k=c["top_k"])
        return nss.route_backward(c["dweights"], c["logits"], c["ids"], h)
    if op == "quantize":
        x = c["x"] if c["batch"] > 1 else c["x"][0]
        q, qt = nss.fp8_quantize(x, c["format"], blocks=c["blocks"], transposed="both", row_index=c.get("index"),
                                 row_div=max(1, c["gather"]))
        out = (q.data, q.scale, qt.data, qt.scale)
        return out if c["batch"] > 1 else tuple(t[None] for t in out)
    if op == "combine":
        return nss.combine(c["o"], c["pos"], c["weights"])
    if op == "combine_gradient":
        return nss.combine_backward(c["dy"], c["o"], c["pos"], c["weights"], do=c["do"])
    if op == "experts_gradient":
        a, b = (nss.Fp8(q, s, q.shape[-1]) for q, s in (c["a"], c["b"]))
        return nss.fp8_matmul_grouped_k(a, b, c["offsets"], out_dtype=TYPES[c["type"]])
    a, b = (nss.Fp8(q, s, c["k"]) for q, s in (c["a"], c["b"]))
    if op == "experts":
        return nss.fp8_matmul(a, b, out=c["out"], offsets=c["offsets"])
    return nss.fp8_matmul(a, b, out_dtype=TYPES[c["type"]])


def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["op"]](state)


# ----------------------------------------------------------------------------- what a pass cannot do without

def work(case):
    c = case
    op = c["op"]
    if op == "route":
        t, k, e = c["tokens"], c["top_k"], c["experts"]
        b = t * e * SIZE[c["type"]] + t * k * (4 + 4 + 4) + 4 * _capacity(t * k, e, c["align"]) + 8 * e
        return {"bytes": b + (4 * e if c["bias"] else 0), "flops": 4 * t * e}
    if op == "route_gradient":
        t, k, e = c["tokens"], c["top_k"], c["experts"]
        return {"bytes": 2 * t * e * SIZE[c["type"]] + 8 * t * k, "flops": 6 * t * e}
    if op == "quantize":
        source = -(-c["rows"] // max(1, c["gather"]))
        n = c["batch"] * c["rows"] * c["cols"]
        q = c["batch"] * (c["rows"] * _up(c["cols"], 128) + c["cols"] * _up(c["rows"], 128))
        return {"bytes": c["batch"] * source * c["cols"] * SIZE[c["type"]] + q + q // 128
                + (4 * c["rows"] if c["gather"] else 0), "flops": 3 * n}
    if op == "product":
        m, n, k = c["m"], c["n"], c["k"]
        return {"bytes": (m + n) * (_up(k, 128) + _up(k, 128) // 128) + m * n * SIZE[c["type"]],
                "flops": 2 * m * n * k}
    rows = c["tokens"] * c["top_k"]
    if op in ("combine", "combine_gradient"):
        e = SIZE[c["type"]] * c["cols"]
        moved = (rows + c["tokens"]) * e + 8 * rows
        return {"bytes": moved + (rows * e + 4 * rows if op == "combine_gradient" else 0), "flops": 4 * rows * c["cols"]}
    weights = c["experts"] * c["n"] * c["k"]
    if op == "experts":
        used = min(1.0, rows / c["experts"])   # a few tokens read the weights of their own experts only
        return {"bytes": int(rows * (c["k"] * 129 / 128 + c["n"] * SIZE[c["type"]]) + used * weights * 129 / 128),
                "flops": 2 * rows * c["n"] * c["k"]}
    return {"bytes": int(rows * (c["k"] + c["n"]) * 129 / 128) + weights * SIZE[c["type"]],
            "flops": 2 * rows * c["n"] * c["k"]}


# ----------------------------------------------------------------------------- exact values, in 64 bits

def _exact_quantize(x, fmt, blocks):
    """Rows of x in double: the scale from logarithms, the values on the format's own grid."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    most = 448.0 if fmt == "e4m3" else 57344.0
    rows, cols = x.shape
    wide = torch.zeros(_up(rows, 128) if blocks else rows, _up(cols, 128), dtype=torch.float64, device=x.device)
    wide[:rows, :cols] = x
    b = wide.view(-1, 128 if blocks else 1, wide.shape[1] // 128, 128)
    amax = b.abs().amax(dim=(1, 3), keepdim=True)
    e = torch.where(amax > 0, torch.ceil(torch.log2(amax / most)), 0.0)
    v = b / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))).clamp(min=low) - bits)
    q = (torch.round(v / step) * step).reshape(wide.shape)[:rows]
    s = torch.ones(rows, _up(wide.shape[1] // 128, 4), dtype=torch.float64, device=x.device)
    s[:, :wide.shape[1] // 128] = torch.exp2(e).expand(-1, b.shape[1], -1, -1).reshape(wide.shape[0], -1)[:rows]
    return q, s


def _exact_values(q, s):
    return q.double() * s.double().repeat_interleave(128, dim=-1)[..., :q.shape[-1]]


def _exact_route(c):
    l = c["logits"].double().cpu().numpy()
    if c["score"] == "softmax":
        s = np.exp(l - l.max(axis=1, keepdims=True))
        s /= s.sum(axis=1, keepdims=True)
    else:
        s = 0.5 * (1.0 + np.tanh(0.5 * l))
    key = s.copy()
    if c["bias_values"] is not None:
        key += c["bias_values"].double().cpu().numpy()
    if c["groups"] > 1:
        per = c["experts"] // c["groups"]
        best = np.sort(key.reshape(len(key), c["groups"], per), axis=2)[:, :, -2:].sum(axis=2)
        out = np.argsort(-best, axis=1, kind="stable")[:, c["top_groups"]:]
        for j in range(out.shape[1]):
            lane = out[:, j:j + 1] * per + np.arange(per)
            np.put_along_axis(key, lane, -np.inf, axis=1)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :c["top_k"]]
    w = np.take_along_axis(s, ids, axis=1)
    return None, torch.from_numpy(w / (w.sum(axis=1, keepdims=True) + 1e-20)), None, None, None, None


def exact(case, seed):
    c = prepare(case, seed)
    op = c["op"]
    if op == "route":
        return _exact_route(c)
    if op == "route_gradient":
        # w_j = s_j / sum of the chosen s; differentiated through log s
        l = c["logits"].double()
        ids, dw = c["ids"].long(), c["dweights"].double()
        logs = torch.log_softmax(l, 1) if c["score"] == "softmax" else -torch.log1p(torch.exp(-l))
        s = torch.exp(logs)
        w = torch.softmax(logs.gather(1, ids), 1)
        dlog = w * (dw - (w * dw).sum(1, keepdim=True))
        full = torch.zeros_like(l)
        full.scatter_(1, ids, dlog)
        if c["score"] == "softmax":
            return full - s * dlog.sum(1, keepdim=True)
        return full * (1.0 - s)
    if op == "quantize":
        got = [[], [], [], []]
        for x in c["x"]:
            x = x.double()
            if c["gather"]:
                i = c["index"].long()
                x = x[i.clamp(min=0).div(c["gather"], rounding_mode="floor")] * (i >= 0)[:, None]
            for j, t in enumerate(_exact_quantize(x, c["format"], c["blocks"]) +
                                  _exact_quantize(x.t(), c["format"], c["blocks"])):
                got[j].append(t)
        return tuple(torch.stack(t) for t in got)
    if op == "product":
        return torch.matmul(_exact_values(*c["a"]), _exact_values(*c["b"]).t())
    if op in ("experts", "experts_gradient"):
        a, off, outs = _exact_values(*c["a"]), c["offsets"].tolist(), []
        if op == "experts":
            y = torch.zeros(len(c["rows_of"]), c["n"], dtype=torch.float64, device=DEV)
            for e in range(c["experts"]):
                y[off[e]:off[e + 1]] = a[off[e]:off[e + 1]] @ _exact_values(c["b"][0][e], c["b"][1][e]).t()
            return y
        b = _exact_values(*c["b"])
        for e in range(c["experts"]):
            outs.append(a[:, off[e]:off[e + 1]] @ b[:, off[e]:off[e + 1]].t())
        return torch.stack(outs)
    o, w, at = c["o"].double(), c["weights"].double(), c["pos"].long()
    if op == "combine":
        y = torch.zeros(c["tokens"], c["cols"], dtype=torch.float64, device=DEV)
        for j in range(c["top_k"]):
            y += w[:, j:j + 1] * o[at[:, j]]
        return y
    dy, do = c["dy"].double(), torch.zeros_like(o)
    dw = torch.zeros_like(w)
    for j in range(c["top_k"]):
        dw[:, j] = (dy * o[at[:, j]]).sum(1)
        do[at[:, j]] = w[:, j:j + 1] * dy
    return dw, do
