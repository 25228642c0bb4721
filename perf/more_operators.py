"""Cases, plain forms and exact values of the operators between a layer's products.

What a training step of a transformer layer needs around its 8-bit products and the Muon
step: the RMS norm with the residual's addition (its output in 8 bits where a product
reads it) and its gradient, attention over packed sequences and its gradient, the
embedding and its gradient, and the clipping of the gradients by their global norm. `own`
chooses between the plain form below and this repository's calls.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
FMT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6


# ----------------------------------------------------------------------------- cases

def listed():
    """Sizes: a 7B-class layer (4096, 11008, 32 heads of 128, 32000 tokens in the vocabulary), a
    smaller one (2048) and the smallest matrices (128, 512), as this repository's workloads have them."""
    return [
        # one step of 16 sequences: latency alone
        {"name": "norm few rows", "op": "norm", "rows": 16, "cols": 4096, "type": "bf16", "weight": "f32",
         "residual": True, "format": ""},
        # a batch in front of an 8-bit projection: the residual stream goes on, the normed rows only in 8 bits
        {"name": "norm to 8 bits", "op": "norm", "rows": 8192, "cols": 4096, "type": "bf16", "weight": "f32",
         "residual": True, "format": "e4m3"},
        # the norm's gradient joined with the residual stream's, an odd number of rows
        {"name": "norm gradient", "op": "norm_gradient", "rows": 16383, "cols": 2048, "type": "bf16", "weight": "f32",
         "residual": True},
        # short texts packed into one batch, every token sees its whole text
        {"name": "attention packed", "op": "attention", "tokens": 4095, "sequences": 32, "cut": 1, "heads": 16,
         "kv_heads": 16, "dim": 64, "causal": False, "window": 0, "type": "f16"},
        # one long text, four heads share a key head
        {"name": "attention long", "op": "attention", "tokens": 8192, "sequences": 1, "cut": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "causal": True, "window": 0, "type": "bf16"},
        # a training batch of packed texts of different lengths
        {"name": "attention gradient packed", "op": "attention_gradient", "tokens": 8191, "sequences": 12, "cut": 2,
         "heads": 32, "kv_heads": 32, "dim": 128, "causal": True, "window": 0, "type": "bf16"},
        # the gradient of the long text
        {"name": "attention gradient long", "op": "attention_gradient", "tokens": 8192, "sequences": 1, "cut": 0,
         "heads": 32, "kv_heads": 8, "dim": 128, "causal": True, "window": 0, "type": "bf16"},
        # the rows of a batch out of the fp32 master embedding
        {"name": "embedding", "op": "embedding", "tokens": 16384, "vocab": 32000, "cols": 4096, "table": "f32",
         "type": "bf16", "scale": 64.0},
        # its gradient for the AdamW step: every row of the vocabulary is written
        {"name": "embedding gradient", "op": "embedding_gradient", "tokens": 16384, "vocab": 32000, "cols": 4096,
         "table": "f32", "type": "bf16", "scale": 64.0, "accumulate": False},
        # a micro-batch added to the gradient so far: only the rows of its tokens are touched
        {"name": "embedding gradient added", "op": "embedding_gradient", "tokens": 1000, "vocab": 32000, "cols": 2048,
         "table": "f32", "type": "bf16", "scale": 1.0, "accumulate": True},
        # many small tensors: launches count
        {"name": "clip small tensors", "op": "clip", "layers": 16, "cols": 128, "inner": 512, "type": "f32",
         "out": "f32", "share": 0.5},
        # an owner's share, accumulated in fp32, clipped into the packed bf16 gradients that the step reads
        {"name": "clip owner share", "op": "clip", "layers": 4, "cols": 4096, "inner": 11008, "type": "f32",
         "out": "bf16", "share": 0.1},
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_gradient", "attention", "attention", "attention_gradient",
                     "attention_gradient", "embedding", "embedding_gradient", "embedding_gradient", "clip"])
    kind = rng.choice(["f32", "bf16", "f16"])
    other = rng.choice(["f32", kind])
    if op in ("norm", "norm_gradient"):
        rows = _spread(rng, 1, 16384)
        c = {"op": op, "rows": rows, "cols": _spread(rng, 8, min(11008, (1 << 26) // rows)), "type": kind,
             "weight": other, "residual": rng.random() < 0.7}
        if op == "norm":
            c["format"] = rng.choice(["", "", "e4m3", "e5m2"])
        return c
    if op in ("attention", "attention_gradient"):
        causal = rng.random() < 0.75
        tokens = _spread(rng, 1, 8192 if causal else 4096)
        kv = rng.choice([1, 2, 4, 5, 8])
        return {"op": op, "tokens": tokens, "sequences": min(tokens, rng.choice([1, 1, _spread(rng, 2, 64)])),
                "cut": rng.randrange(1000), "heads": kv * rng.choice([1, 2, 3, 4]), "kv_heads": kv,
                "dim": rng.choice([64, 64, 128, 128, 128, 32, 40, 72, 96, 120]), "causal": causal,
                "window": _spread(rng, 1, 4096) if causal and rng.random() < 0.3 else 0,
                "type": rng.choice(["bf16", "bf16", "f16"])}
    if op in ("embedding", "embedding_gradient"):
        c = {"op": op, "tokens": _spread(rng, 1, 16384), "vocab": _spread(rng, 128, 32000), "cols": _spread(rng, 16, 4096),
             "table": other, "type": kind, "scale": rng.choice([1.0, 8.0])}
        if op == "embedding_gradient":
            c["accumulate"] = rng.random() < 0.5
        return c
    return {"op": op, "layers": rng.randint(1, 32), "cols": _spread(rng, 64, 1024), "inner": _spread(rng, 100, 2048),
            "type": kind, "out": other, "share": rng.choice([0.01, 0.5, 3.0])}


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


def _lengths(c):
    """Lengths of the packed sequences, the longest under twice the mean; from four sequences on
    one is empty and one has a single token. They go by the case alone, so that its work does."""
    n, tokens = c["sequences"], c["tokens"]
    r = np.random.RandomState(c["cut"])
    w = 0.3 + r.rand(n)
    if n >= 4:
        w[1] = w[2] = 0.0
    got = np.floor((tokens - (n >= 4)) * w / w.sum()).astype(np.int64)
    if n >= 4:
        got[2] = 1
    got[n - 1] += tokens - got.sum()
    return got


def _shapes(c):
    """The tensors of `layers` layers: four square matrices, three wide ones, two vectors."""
    n, m = c["cols"], c["inner"]
    return ([(n, n)] * 4 + [(m, n), (m, n), (n, m), (n,), (n,)]) * c["layers"]


def _ids(g, c):
    """Token ids as texts have them: the k-th most frequent one about 1/k as often; 2% padding (-1)."""
    u = torch.rand(c["tokens"], generator=g, device=DEV, dtype=torch.float64)
    ids = (torch.exp(u * math.log(c["vocab"])).long() - 1).clamp(0, c["vocab"] - 1)
    ids = torch.randperm(c["vocab"], generator=g, device=DEV)[ids]
    return torch.where(torch.rand(c["tokens"], generator=g, device=DEV) < 0.02, -1, ids).to(torch.int32)


def prepare(case, seed):
    g, c = _generator(seed), dict(case)
    op, kind = c["op"], TYPES[c["type"]]
    if op in ("norm", "norm_gradient"):
        rows, cols = c["rows"], c["cols"]
        c["x"] = _activations(g, rows, cols).to(kind)
        c["w"] = (1.0 + 0.1 * _normal(g, cols)).to(TYPES[c["weight"]])
        if op == "norm":
            c["r"] = (2.0 * _activations(g, rows, cols)).to(kind) if c["residual"] else None
        else:
            c["rstd"] = torch.rsqrt(c["x"].float().square().mean(1) + EPS)
            c["dy"] = (0.01 * _normal(g, rows, cols)).to(kind)
            c["ds"] = (0.01 * _normal(g, rows, cols)).to(kind) if c["residual"] else None
    elif op in ("attention", "attention_gradient"):
        t, d = c["tokens"], c["dim"]
        loud = torch.exp(0.3 * _normal(g, c["heads"], 1))   # some heads look more sharply
        c["q"] = (_normal(g, t, c["heads"], d) * loud).to(kind)
        c["k"] = _normal(g, t, c["kv_heads"], d).to(kind)
        c["v"] = _normal(g, t, c["kv_heads"], d).to(kind)
        n = _lengths(c)
        c["most"] = int(n.max())
        c["offsets"] = torch.from_numpy(np.concatenate([[0], n.cumsum()]).astype(np.int32)).to(DEV)
        if op == "attention_gradient":
            c["o"], c["lse"] = _run_attention(c)
            c["do"] = (0.1 * _normal(g, t, c["heads"], d)).to(kind)
    elif op in ("embedding", "embedding_gradient"):
        c["ids"] = _ids(g, c)
        if op == "embedding":
            c["w"] = (0.02 * _normal(g, c["vocab"], c["cols"])).to(TYPES[c["table"]])
        else:
            c["dy"] = (0.01 * _normal(g, c["tokens"], c["cols"])).to(kind)
            if c["accumulate"]:
                c["dw"] = (0.01 * _normal(g, c["vocab"], c["cols"])).to(TYPES[c["table"]])
    else:
        shapes = _shapes(c)
        c["grads"] = [(0.01 * _normal(g, *s)).to(kind) for s in shapes]
        sizes = [math.prod(s) for s in shapes]
        c["max_norm"] = c["share"] * 0.01 * math.sqrt(sum(sizes))
        starts = np.cumsum([0] + [_up(n, 64) for n in sizes])
        c["packed"] = torch.zeros(int(starts[-1]), dtype=TYPES[c["out"]], device=DEV)
        c["outs"] = [c["packed"][b:b + n].view(s) for b, n, s in zip(starts.tolist(), sizes, shapes)]
    return c


# ----------------------------------------------------------------------------- plain forms

def _to_8_bits(y, fmt):
    """Rows in blocks of 128 with a power-of-two scale that their largest value just fits."""
    y = torch.nn.functional.pad(y.float(), (0, -y.shape[1] % 128)).unflatten(1, (-1, 128))
    half, e = torch.frexp(y.abs().amax(2) / LARGEST[fmt])       # half in [0.5, 1)
    e = torch.where(half > 0, torch.where(half == 0.5, e - 1, e).clamp(min=-126), 0).to(torch.int32)
    q = (y * ((127 - e) << 23).view(torch.float32)[:, :, None]).flatten(1).to(FMT[fmt])
    s = torch.nn.functional.pad(e, (0, -e.shape[1] % 4)) + 127
    return q, s.to(torch.uint8).view(torch.float8_e8m0fnu)


def _run_norm(c):
    x = c["x"]
    s = x if c["r"] is None else (x.float() + c["r"].float()).to(x.dtype)
    f = s.float()
    rstd = torch.rsqrt(f.square().mean(1) + EPS)
    y = (f * rstd[:, None] * c["w"].float()).to(x.dtype)
    return (s, rstd) + (_to_8_bits(y, c["format"]) if c["format"] else (y,))


def _run_norm_gradient(c):
    s, dy, rstd = c["x"].float(), c["dy"].float(), c["rstd"][:, None]
    n = s * rstd
    g = dy * c["w"].float()
    dx = rstd * (g - n * (g * n).mean(1, keepdim=True))
    if c["ds"] is not None:
        dx = dx + c["ds"].float()
    return dx.to(c["x"].dtype), (dy * n).sum(0)


def _places(c):
    """Rows of the sequences padded to the longest, [sequences, most], and which of them are there."""
    at = c["offsets"][:-1, None].long() + torch.arange(c["most"], device=DEV)
    return at.clamp(max=c["tokens"] - 1), at < c["offsets"][1:, None]


def _padded(x, at, has):
    """[tokens, heads, dim] -> [sequences, heads, most, dim] in 32 bits, zeros behind the ends."""
    return (x[at].float() * has[:, :, None, None]).transpose(1, 2).contiguous()


def _grouped(x, c):
    """[.., heads, most, dim] -> [.., key heads, heads of the group x most, dim]"""
    return x.unflatten(1, (c["kv_heads"], -1)).flatten(2, 3)


def _scores(c, q, k, has):
    """[sequences, key heads, heads of the group, most, most], -inf where a key is not seen."""
    s = torch.matmul(_grouped(q, c), k.transpose(2, 3).contiguous()) * c["dim"] ** -0.5
    i = torch.arange(c["most"], device=DEV)
    seen = has[:, None, :] & has[:, :, None]
    if c["causal"]:
        seen = seen & (i[:, None] >= i)
    if c["window"]:
        seen = seen & (i[:, None] - i < c["window"])
    seen = seen | (~has[:, :, None] & (i == 0))    # rows behind the ends: anything but NaN
    return s.unflatten(2, (-1, c["most"])).masked_fill_(~seen[:, None, None], -math.inf)


def _packed(x, c, has):
    """[sequences, key heads, group x most, dim] -> [tokens, heads, dim]"""
    return x.unflatten(2, (-1, c["most"])).flatten(1, 2).transpose(1, 2)[has]


def _run_attention(c):
    at, has = _places(c)
    s = _scores(c, _padded(c["q"], at, has), _padded(c["k"], at, has), has)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s.sub_(top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), _padded(c["v"], at, has)) / total.flatten(2, 3)
    lse = (top + torch.log(total)).flatten(1, 2)[..., 0]
    return _packed(o, c, has).to(c["q"].dtype), lse.transpose(1, 2)[has].t().contiguous()


def _run_attention_gradient(c):
    at, has = _places(c)
    q, k, v = (_padded(c[n], at, has) for n in "qkv")
    do, o = (_padded(c[n], at, has) for n in ("do", "o"))
    lse = _padded(c["lse"].t().contiguous()[:, :, None], at, has).unflatten(1, (c["kv_heads"], -1))
    p = torch.exp(_scores(c, q, k, has) - lse).flatten(2, 3)
    g = _grouped(do, c)
    dv = torch.matmul(p.transpose(2, 3).contiguous(), g)
    ds = torch.matmul(g, v.transpose(2, 3).contiguous())
    ds = ds.sub_(_grouped((do * o).sum(-1, keepdim=True), c)).mul_(p).mul_(c["dim"] ** -0.5)
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(2, 3).contiguous(), _grouped(q, c))
    kind = c["q"].dtype
    return _packed(dq, c, has).to(kind), dk.transpose(1, 2)[has].to(kind), dv.transpose(1, 2)[has].to(kind)


def _run_embedding(c):
    rows = c["w"][c["ids"].clamp(min=0)].float() * c["scale"]
    return torch.where(c["ids"][:, None] >= 0, rows, 0.0).to(TYPES[c["type"]])


def _run_embedding_gradient(c):
    is_token = c["ids"] >= 0
    rows = torch.where(is_token[:, None], c["dy"].float() * c["scale"], 0.0)
    total = torch.zeros(c["vocab"], c["cols"], device=DEV).index_add_(0, c["ids"].clamp(min=0), rows)
    if c["accumulate"]:
        return c["dw"].copy_(c["dw"].float() + total)
    return total.to(TYPES[c["table"]])


def _run_clip(c):
    norm = torch.stack([g.double().square().sum() for g in c["grads"]]).sum().sqrt()
    factor = (c["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    [o.copy_(g.float() * factor) for o, g in zip(c["outs"], c["grads"])]
    return c["packed"], norm.float()


PLAIN = {"norm": _run_norm, "norm_gradient": _run_norm_gradient, "attention": _run_attention,
         "attention_gradient": _run_attention_gradient, "embedding": _run_embedding,
         "embedding_gradient": _run_embedding_gradient, "clip": _run_clip}


# ----------------------------------------------------------------------------- this repository's calls

def _run_own(c):
    import newton_schulz_step_amd as nss
    op = c["op"]
    if op == "norm":
        n = nss.rms_norm(c["x"], c["w"], residual=c["r"], eps=EPS, fp8="only" if c["format"] else "no",
                         fmt=c["format"] or "e4m3")
        return (n.sum, n.rstd) + ((n.fp8.data, n.fp8.scale) if c["format"] else (n.y,))
    if op == "norm_gradient":
        return nss.rms_norm_backward(c["dy"], c["x"], c["w"], c["rstd"], dsum=c["ds"])
    if op in ("attention", "attention_gradient"):
        how = {"offsets": c["offsets"] if c["sequences"] > 1 else None, "causal": c["causal"], "window": c["window"]}
        if op == "attention":
            return nss.attention(c["q"], c["k"], c["v"], **how)
        return nss.attention_backward(c["do"], c["q"], c["k"], c["v"], c["o"], c["lse"], **how)
    if op == "embedding":
        return nss.embedding(c["ids"], c["w"], scale=c["scale"], out_dtype=TYPES[c["type"]])
    if op == "embedding_gradient":
        return nss.embedding_backward(c["dy"], c["ids"], c["vocab"], scale=c["scale"], out=c.get("dw"),
                                      out_dtype=TYPES[c["table"]], accumulate=c["accumulate"])
    norm = nss.clip_gradients(c["grads"], c["max_norm"], out=c["outs"])
    return c["packed"], norm


def run(state):
    if own:
        return _run_own(state)
    return PLAIN[state["op"]](state)


# ----------------------------------------------------------------------------- what a pass cannot do without

def _pairs(c):
    """Keys seen, summed over the rows of all sequences."""
    n = _lengths(c)
    w = np.minimum(n, c["window"] or n)
    return int((w * (w + 1) // 2 + (n - w) * w).sum() if c["causal"] else (n * n).sum())


def _distinct(c):
    """How many different tokens a batch is expected to hold."""
    k = np.arange(1, c["vocab"] + 1)
    p = np.log1p(1.0 / k) / math.log(c["vocab"] + 1)
    return int((1.0 - (1.0 - p) ** c["tokens"]).sum())


def work(case):
    c = case
    op, e = c["op"], SIZE[c["type"]]
    if op in ("norm", "norm_gradient"):
        n = c["rows"] * c["cols"]
        if op == "norm":
            moved = (3 if c["residual"] else 1) * n * e
            moved += c["rows"] * _up(c["cols"], 128) * 129 // 128 if c["format"] else n * e
        else:
            moved = (4 if c["residual"] else 3) * n * e + 4 * c["cols"]
        return {"bytes": moved + c["cols"] * SIZE[c["weight"]] + 4 * c["rows"], "flops": (4 if op == "norm" else 9) * n}
    if op in ("attention", "attention_gradient"):
        q, kv = (c["tokens"] * c[h] * c["dim"] * e for h in ("heads", "kv_heads"))
        lse, products = 4 * c["tokens"] * c["heads"], 2 * _pairs(c) * c["heads"] * c["dim"]
        if op == "attention":
            return {"bytes": 2 * q + 2 * kv + lse, "flops": 2 * products}
        return {"bytes": 4 * q + 4 * kv + lse, "flops": 5 * products}
    if op in ("embedding", "embedding_gradient"):
        n, table = c["tokens"] * c["cols"], c["cols"] * SIZE[c["table"]]
        if op == "embedding":
            return {"bytes": n * e + 4 * c["tokens"] + _distinct(c) * table, "flops": n}
        rows = 2 * _distinct(c) if c["accumulate"] else c["vocab"]
        return {"bytes": n * e + 4 * c["tokens"] + rows * table, "flops": 2 * n}
    n = sum(math.prod(s) for s in _shapes(c))
    return {"bytes": n * (e + SIZE[c["out"]]), "flops": 3 * n}


# ----------------------------------------------------------------------------- exact values, in 64 bits

def _exact_8_bits(y, fmt):
    """Rows in double: the scale from logarithms, the values on the format's own grid."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    rows, cols = y.shape
    b = torch.zeros(rows, _up(cols, 128), dtype=torch.float64, device=DEV)
    b[:, :cols] = y
    b = b.view(rows, -1, 128)
    most = b.abs().amax(2, keepdim=True)
    scale = torch.exp2(torch.where(most > 0, torch.ceil(torch.log2(most / LARGEST[fmt])), 0.0))
    v = b / scale
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** low))).clamp(min=low) - bits)
    s = torch.ones(rows, _up(b.shape[1], 4), dtype=torch.float64, device=DEV)
    s[:, :b.shape[1]] = scale[:, :, 0]
    return (torch.round(v / step) * step).view(rows, -1), s


def _exact_heads(c, f):
    """f(queries of the group, keys, values, first row, first head, mask) for each key head of each sequence."""
    group, start = c["heads"] // c["kv_heads"], 0
    for n in _lengths(c).tolist():
        i = torch.arange(n, device=DEV)
        far = i[:, None] - i
        hidden = torch.zeros(n, n, dtype=torch.bool, device=DEV)
        if c["causal"]:
            hidden |= far < 0
        if c["window"]:
            hidden |= far >= c["window"]
        for h in range(c["heads"] if n else 0):
            q, k, v = c["q"][start:start + n, h], c["k"][start:start + n, h // group], c["v"][start:start + n, h // group]
            s = q.double() @ k.double().t() / math.sqrt(c["dim"])
            f(slice(start, start + n), h, h // group, s.masked_fill(hidden, -math.inf), q.double(), k.double(), v.double())
        start += n


def _exact_attention(c):
    o = torch.zeros(c["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(c["heads"], c["tokens"], dtype=torch.float64, device=DEV)

    def one(rows, h, _, s, q, k, v):
        lse[h, rows] = torch.logsumexp(s, 1)
        o[rows, h] = torch.softmax(s, 1) @ v

    _exact_heads(c, one)
    return o, lse


def _exact_attention_gradient(c):
    dq, dk, dv = (torch.zeros(c[n].shape, dtype=torch.float64, device=DEV) for n in "qkv")

    def one(rows, h, kv, s, q, k, v):
        p, g = torch.softmax(s, 1), c["do"][rows, h].double()
        dv[rows, kv] += p.t() @ g
        dp = g @ v.t()
        ds = p * (dp - (p * dp).sum(1, keepdim=True)) / math.sqrt(c["dim"])
        dq[rows, h] = ds @ k
        dk[rows, kv] += ds.t() @ q

    _exact_heads(c, one)
    return dq, dk, dv


def exact(case, seed):
    c = prepare(case, seed)
    op, kind = c["op"], TYPES[c["type"]]
    if op == "norm":
        total = c["x"].double() if c["r"] is None else c["x"].double() + c["r"].double()
        s = total.to(kind).double()
        rms = ((s * s).sum(1) / c["cols"] + EPS).sqrt()
        y = s / rms[:, None] * c["w"].double()
        return (total, 1.0 / rms) + (_exact_8_bits(y.to(kind).double(), c["format"]) if c["format"] else (y,))
    if op == "norm_gradient":
        # y = x w / rms, rms^2 = x.x / n + eps: dx = (w dy) / rms - x (x . w dy) / (n rms^3)
        x, dy, w = c["x"].double(), c["dy"].double(), c["w"].double()
        rms = ((x * x).sum(1, keepdim=True) / c["cols"] + EPS).sqrt()
        dx = w * dy / rms - x * ((x * w * dy).sum(1, keepdim=True) / (c["cols"] * rms ** 3))
        return dx if c["ds"] is None else dx + c["ds"].double(), (dy * x / rms).sum(0)
    if op == "attention":
        return _exact_attention(c)
    if op == "attention_gradient":
        return _exact_attention_gradient(c)
    if op == "embedding":
        padded = torch.cat([c["w"].double(), torch.zeros(1, c["cols"], dtype=torch.float64, device=DEV)])
        return c["scale"] * padded[c["ids"].long()]          # id -1 is the last row, of zeros
    if op == "embedding_gradient":
        dw = torch.zeros(c["vocab"] + 1, c["cols"], dtype=torch.float64, device=DEV)
        dw.index_put_((c["ids"].long(),), c["scale"] * c["dy"].double(), accumulate=True)
        return dw[:-1] + c["dw"].double() if c["accumulate"] else dw[:-1]
    norm = math.sqrt(sum(float(torch.linalg.vector_norm(g.double())) ** 2 for g in c["grads"]))
    packed = torch.zeros(c["packed"].shape, dtype=torch.float64, device=DEV)
    start = 0
    for g in c["grads"]:
        packed[start:start + g.numel()] = g.double().view(-1) * min(1.0, c["max_norm"] / (norm + 1e-6))
        start += _up(g.numel(), 64)
    return packed, norm
