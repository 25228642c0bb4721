"""GPU: attention over packed sequences and its gradient against the float64 oracle.

The tolerances bound what the kernels round, per value. U = 2^-24 (fp32), HALF = half a step
of the operands' type.
  a score: its products are exact in fp32, dim of them are summed, then scaled: a relative
    error of the exponential of d = U (dim + 8) scale sum |q k| + 4 U, and of U |lse| more
    where the stored log-sum-exp is used
  a probability, rounded as a product's operand: HALF
  sums over n keys or rows: U n
  fp16 operands below 2^-14 of the scale they carry: 2^-25 of it, absolutely (row maximum
    in the forward pass; 2^-8 and 2^-10 of the column's largest in the gradient)
  below the smallest normal number of fp32 and bf16 (LOW = 2^-126) the exponential and the
    matrix instructions may give 0: LOW per probability and score gradient (a probability of
    2^-127 times dP of 10 is a score gradient of 2^-124 that is lost whole), and LOW per step
    of a sum
"""
import numpy as np
import pytest

from oracle import layer as L

pytestmark = pytest.mark.gpu

HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -24}
U = 2.0 ** -24
LOW = 2.0 ** -126


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def host(t):
    return t.detach().cpu().double().numpy()


def offsets_of(lens):
    import torch
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda")


def make(seed, tokens, heads, kv, dim, dtype, loud=1.0, grad=0.1):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(h, k):
        return (k * torch.randn(tokens, h, dim, generator=g, device="cuda")).to(dt(dtype))
    return n(heads, loud), n(kv, 1.0), n(kv, 1.0), n(heads, grad)


def check_forward(q, k, v, out, lse, dtype, **how):
    q, k, v, out, lse = (host(t) for t in (q, k, v, out, lse))
    scale = how.get("scale") or q.shape[2] ** -0.5
    half, dim = HALF[dtype], q.shape[2]
    for rows, h, kv, s, p, l in L.attention_heads(q, k, v, **how):
        n = s.shape[0]
        d = U * (dim + 8) * scale * np.max(np.where(np.isfinite(s), np.abs(q[rows, h]) @ np.abs(k[rows, kv]).T, 0), axis=1) + 4 * U
        want = p @ v[rows, kv]
        mag = p @ np.abs(v[rows, kv])
        tol = half * (mag + np.abs(want)) + (2 * d + U * (n + 16))[:, None] * mag + LOW * (n + np.sum(np.abs(v[rows, kv]), axis=0)) + TINY[dtype]
        if dtype == "f16":
            tol = tol + 2.0 ** -25 * np.where(np.isfinite(s), 1.0, 0.0) @ np.abs(v[rows, kv])
        err = np.abs(out[rows, h] - want)
        assert np.all(err <= tol), (h, np.max(err / tol), np.unravel_index(np.argmax(err / tol), err.shape))
        err, tol = np.abs(lse[h, rows] - l), d + U * (n + 16) + 4 * U * np.abs(l)
        assert np.all(err <= tol), ("lse", h, np.max(err / tol))


def check_backward(do, q, k, v, out, got, dtype, **how):
    do, q, k, v, out = (host(t) for t in (do, q, k, v, out))
    got = [host(t) for t in got]
    scale = how.get("scale") or q.shape[2] ** -0.5
    half, dim = HALF[dtype], q.shape[2]
    want = L.attention_backward(do, q, k, v, **how)
    tol = [half * np.abs(w) + TINY[dtype] + LOW * len(q) for w in want]
    for rows, h, kv, s, p, l in L.attention_heads(q, k, v, **how):
        n = s.shape[0]
        seen = np.isfinite(s)
        qq, kk, vv, g, o = q[rows, h], k[rows, kv], v[rows, kv], do[rows, h], out[rows, h]
        d = U * (dim + 8) * scale * np.max(np.where(seen, np.abs(qq) @ np.abs(kk).T, 0), axis=1) + 8 * U + 4 * U * np.abs(l)
        e = (2 * d + U * (n + 16))[:, None]
        dp = g @ vv.T
        delta = np.sum(p * dp, axis=1, keepdims=True)
        # delta comes from the rounded output
        gd = half * np.sum(np.abs(g) * np.abs(o), axis=1, keepdims=True) + U * (dim + 8) * np.sum(np.abs(g) * np.abs(o), axis=1, keepdims=True)
        ds = p * (dp - delta)
        es = p * (gd + U * (dim + 4) * (np.abs(g) @ np.abs(vv).T)) + (half + e) * np.abs(ds) + e * p * (np.abs(dp) + np.abs(delta))
        ep = (half + e) * p + LOW * seen
        es = es + LOW * seen * (1 + np.abs(dp) + np.abs(delta))
        if dtype == "f16":
            es = es + 2.0 ** -34 * np.where(seen, max(np.max(np.abs(ds)), 0), 0)
            ep = ep + 2.0 ** -33 * seen
        tol[0][rows, h] += scale * (es + U * n * np.abs(ds)) @ np.abs(kk)
        tol[1][rows, kv] += scale * (es + U * (n + 64) * np.abs(ds)).T @ np.abs(qq)
        tol[2][rows, kv] += (ep + U * (n + 64) * p).T @ np.abs(g)
    for name, x, w, t in zip(("dq", "dk", "dv"), got, want, tol):
        inside = np.zeros(x.shape, bool)
        for b, e in L._sequences(how.get("offsets"), x.shape[0]):
            inside[b:e] = True
        err = np.where(inside, np.abs(x - w), 0)
        assert np.all(err <= t), (name, np.max(err / t), np.unravel_index(np.argmax(err / t), err.shape))


LENS = [[1], [2], [31, 33], [64], [65], [127, 1, 0, 128], [129], [200, 0, 1, 77, 300], [513], [0, 0, 5], [1] * 70, [700]]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [8, 32, 40, 64, 72, 96, 104, 128])
@pytest.mark.parametrize("lens", LENS, ids=lambda l: f"{len(l)}x{max(l)}")
def test_forward_and_gradient(lib, lens, dim, dtype):
    tokens = int(np.sum(lens))
    shapes = [(4, 2, True, 0), (3, 3, False, 0), (8, 1, True, 50)] if tokens < 400 else [(8, 2, True, 0), (2, 2, False, 0), (2, 1, True, 130)]
    for heads, kv, causal, window in shapes:
        q, k, v, do = make(dim + tokens, tokens, heads, kv, dim, dtype, loud=2.0)
        off = offsets_of(lens) if len(lens) > 1 else None
        hoff = None if off is None else off.cpu().numpy()
        how = dict(causal=causal, window=window)
        out, lse = lib.attention(q, k, v, offsets=off, **how)
        check_forward(q, k, v, out, lse, dtype, offsets=hoff, **how)
        got = lib.attention_backward(do, q, k, v, out, lse, offsets=off, **how)
        check_backward(do, q, k, v, out, got, dtype, offsets=hoff, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [24, 40, 64, 80, 128])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 40)])
def test_many_key_tiles(lib, causal, window, dim, dtype):
    """From 1024 key tiles on dK and dV take workgroups of four waves, without parts."""
    lens = [1] * 60 + [130, 0, 33, 64, 200]
    off, hoff = offsets_of(lens), np.cumsum([0] + lens)
    q, k, v, do = make(dim, sum(lens), 32, 16, dim, dtype, loud=2.0)
    assert (sum(lens) // 128 + len(lens)) * 16 >= 1024
    how = dict(causal=causal, window=window)
    out, lse = lib.attention(q, k, v, offsets=off, **how)
    check_forward(q, k, v, out, lse, dtype, offsets=hoff, **how)
    got = lib.attention_backward(do, q, k, v, out, lse, offsets=off, **how)
    check_backward(do, q, k, v, out, got, dtype, offsets=hoff, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_parts_of_few_key_tiles(lib, dtype):
    """Few key tiles: their queries are summed in parts, some of which hold no row that sees a key."""
    for tokens, heads, kv, how in ((1300, 8, 1, {}), (600, 16, 1, dict(window=70)), (520, 4, 2, dict(causal=False))):
        q, k, v, do = make(tokens, tokens, heads, kv, 64, dtype)
        out, lse = lib.attention(q, k, v, **how)
        check_backward(do, q, k, v, out, lib.attention_backward(do, q, k, v, out, lse, **how), dtype, **how)


def test_far_offsets(lib):
    """Elements beyond 2^31 of one tensor."""
    import torch
    stride = 1 << 22
    base = torch.empty(700 * stride, dtype=torch.bfloat16, device="cuda")   # 5.9 GB
    q, k, v, do = make(5, 700, 2, 2, 64, "bf16")

    def far(x, at):
        t = base.as_strided(x.shape, (stride, 64, 1), at)
        t.copy_(x)
        return t
    out, lse = lib.attention(q, k, v)
    want = lib.attention_backward(do, q, k, v, out, lse)
    fo = base.as_strided(q.shape, (stride, 64, 1), 4096)
    fq, fk, fv, fdo = (far(x, 512 * i) for i, x in enumerate((q, k, v, do)))
    _, flse = lib.attention(fq, fk, fv, out=fo)
    assert torch.equal(fo, out) and torch.equal(flse, lse)
    grads = [base.as_strided(q.shape, (stride, 64, 1), 8192 + 512 * i) for i in range(3)]
    lib.attention_backward(fdo, fq, fk, fv, fo, flse, dq=grads[0], dk=grads[1], dv=grads[2])
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 200, 5000])
def test_windows(lib, window, dtype):
    q, k, v, do = make(window, 450, 2, 2, 64, dtype)
    out, lse = lib.attention(q, k, v, window=window)
    check_forward(q, k, v, out, lse, dtype, window=window)
    if window == 1:   # a token sees itself alone
        assert (out == v).all()
    got = lib.attention_backward(do, q, k, v, out, lse, window=window)
    check_backward(do, q, k, v, out, got, dtype, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scale_and_sharp_rows(lib, dtype):
    """Scores far apart (one key takes all, or exponents leave fp32), and other scales."""
    for loud, scale in ((30.0, None), (1.0, 3.0), (1.0, 1e-3), (300.0, 0.5)):
        q, k, v, do = make(3, 300, 4, 2, 64, dtype, loud=loud)
        s = None if scale is None else float(np.float32(scale))
        out, lse = lib.attention(q, k, v, scale=s)
        check_forward(q, k, v, out, lse, dtype, scale=s)
        got = lib.attention_backward(do, q, k, v, out, lse, scale=s)
        check_backward(do, q, k, v, out, got, dtype, scale=s)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [1e-6, 1e-3, 30.0, 6e4])
def test_gradient_range(lib, size, dtype):
    """Output gradients at either end of fp16's range, and rows and heads of very different size."""
    import torch
    q, k, v, _ = make(8, 330, 4, 2, 128, dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    do = torch.rand(330, 4, 128, generator=g, device="cuda") * 2 - 1
    do = (do * size * torch.exp2(-10 * torch.rand(330, 4, 1, generator=g, device="cuda"))).to(dt(dtype))
    out, lse = lib.attention(q, k, v)
    check_backward(do, q, k, v, out, lib.attention_backward(do, q, k, v, out, lse), dtype)


def test_layouts_and_rows_outside(lib):
    """Parts of a joint projection, head-major operands, results into parts of one gradient;
    tokens outside the sequences are not read and their rows not written."""
    import torch
    T, H, K, D = 333, 6, 2, 72
    off = torch.tensor([10, 110, 110, 300], dtype=torch.int32, device="cuda")
    q, k, v, do = make(4, T, H, K, D, "bf16")
    want, want_lse = lib.attention(q, k, v, offsets=off)
    grads = lib.attention_backward(do, q, k, v, want, want_lse, offsets=off)
    check_forward(q[10:300], k[10:300], v[10:300], want[10:300], want_lse[:, 10:300], "bf16", offsets=[0, 100, 100, 290])
    inside = torch.zeros(T, dtype=torch.bool, device="cuda")
    inside[10:300] = True

    joint = torch.full((T, (H + 2 * K) * D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    parts = joint.as_strided((T, H + 2 * K, D), (joint.stride(0), D, 1))
    jq, jk, jv = parts[:, :H], parts[:, H:H + K], parts[:, H + K:]
    for to, x in ((jq, q), (jk, k), (jv, v)):
        to[inside] = x[inside]   # NaN elsewhere
    out = torch.full((H, T, D), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)   # head-major
    lse = torch.full((H, T), 7.0, device="cuda")
    lib.attention(jq, jk, jv, offsets=off, out=out, lse=lse)
    assert torch.equal(out[inside], want[inside]) and torch.equal(lse[:, inside], want_lse[:, inside])
    assert (out[~inside] == 7).all() and (lse[:, ~inside] == 7).all()
    djoint = torch.full_like(joint, 5.0)
    dparts = djoint.as_strided((T, H + 2 * K, D), (djoint.stride(0), D, 1))
    dq, dk, dv = dparts[:, :H], dparts[:, H:H + K], dparts[:, H + K:]
    hdo = do.transpose(0, 1).contiguous().transpose(0, 1)
    lib.attention_backward(hdo, jq, jk, jv, out, lse, offsets=off, dq=dq, dk=dk, dv=dv)
    for x, y in zip((dq, dk, dv), grads):
        assert torch.equal(x[inside], y[inside]) and (x[~inside] == 5).all()
    assert (djoint[:, (H + 2 * K) * D:] == 5).all()
    # one key head for all tokens' heads, expanded
    wide = k[:, :1].expand(T, K, D)
    assert torch.equal(lib.attention(q, wide, v)[0], lib.attention(q, wide.contiguous(), v)[0])


@pytest.mark.parametrize("T", [1, 77])
def test_joint_projection_by_head(lib, T):
    """q, k and v of every head next to each other, and so their gradients."""
    import torch
    H, D = 8, 64
    q, k, v, do = make(8, T, H, H, D, "bf16")
    out, lse = lib.attention(q, k, v)
    grads = lib.attention_backward(do, q, k, v, out, lse)
    joint = torch.stack((q, k, v), dim=2)   # [T, H, 3, D]
    parts = [joint[:, :, i] for i in range(3)]
    assert all(torch.equal(x, y) for x, y in zip(lib.attention(*parts), (out, lse)))
    djoint = torch.full_like(joint, 5.0)
    lib.attention_backward(do, *parts, out, lse, dq=djoint[:, :, 0], dk=djoint[:, :, 1], dv=djoint[:, :, 2])
    for i in range(3):
        assert torch.equal(djoint[:, :, i], grads[i])


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 40)])
@pytest.mark.parametrize("sequences", [1, 2, 63, 64, 65, 200, 1100])
def test_number_of_sequences(lib, sequences, causal, window):
    """Tiles are found in each wave for up to 64 sequences, listed beforehand for more: the same rows with empty
    sequences in between are the same work."""
    import torch
    rng = np.random.default_rng(sequences)
    lens = rng.integers(0, max(3, 1500 // sequences), sequences)
    lens[sequences // 2] = 300
    T = int(lens.sum()) + 6
    off = np.concatenate([[3], 3 + np.cumsum(lens)])
    q, k, v, do = make(sequences, T, 3, 1, 40, "bf16")
    how = dict(causal=causal, window=window)

    def run(at):
        at = torch.from_numpy(np.asarray(at, np.int32)).to("cuda")
        kept = [torch.full_like(t, 9.0) for t in (q, q, k, k)]
        lse = torch.full((3, T), 9.0, device="cuda")
        lib.attention(q, k, v, offsets=at, out=kept[0], lse=lse, **how)
        lib.attention_backward(do, q, k, v, kept[0], lse, offsets=at, dq=kept[1], dk=kept[2], dv=kept[3], **how)
        return kept, lse
    kept, lse = run(off)
    assert all((t[:3] == 9).all() and (t[T - 3:] == 9).all() for t in kept)
    at = slice(3, T - 3)
    check_forward(q[at], k[at], v[at], kept[0][at], lse[:, at], "bf16", offsets=off - 3, **how)
    check_backward(do[at], q[at], k[at], v[at], kept[0][at], [t[at] for t in kept[1:]], "bf16", offsets=off - 3, **how)
    other, other_lse = run(np.concatenate([off, np.full(70, off[-1] - 2)]))   # they fall: empty
    assert torch.equal(lse, other_lse) and all(torch.equal(x, y) for x, y in zip(kept[:2], other[:2]))


def test_offsets_out_of_order_and_range(lib):
    import torch
    q, k, v, do = make(6, 260, 2, 2, 64, "bf16")
    odd = torch.tensor([-5, 100, 40, 160, 1000, 3], dtype=torch.int32, device="cuda")
    plain = torch.tensor([0, 100, 100, 160, 260, 260], dtype=torch.int32, device="cuda")
    a, b = lib.attention(q, k, v, offsets=odd), lib.attention(q, k, v, offsets=plain)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, y in zip(lib.attention_backward(do, q, k, v, *a, offsets=odd), lib.attention_backward(do, q, k, v, *b, offsets=plain)):
        assert torch.equal(x, y)


def test_packed_equals_alone(lib):
    """A sequence's results do not depend on what it is packed with, nor on NaN next to it."""
    import torch
    lens = [150, 64, 1, 333]
    q, k, v, do = make(12, sum(lens), 4, 2, 128, "bf16")
    at = np.cumsum([0] + lens)
    for t in (q, k, v, do):
        t[at[1]:at[2]] = float("nan")
    off = offsets_of(lens)
    out, lse = lib.attention(q, k, v, offsets=off)
    grads = lib.attention_backward(do, q, k, v, out, lse, offsets=off)
    for i in (0, 2, 3):
        r = slice(int(at[i]), int(at[i + 1]))
        o, l = lib.attention(q[r], k[r], v[r])
        assert torch.equal(o, out[r]) and torch.equal(l, lse[:, r])
        assert torch.equal(lib.attention_backward(do[r], q[r], k[r], v[r], o, l)[0], grads[0][r])
        # dk and dv may be summed in other parts
        check_backward(do[r], q[r], k[r], v[r], o, [x[r] for x in grads], "bf16")
    assert torch.isnan(out[at[1]:at[2]]).all()


def test_gradient_against_differences(lib):
    """The slope of <do, out> along a direction, from differences of the oracle in 64 bits."""
    rng = np.random.default_rng(0)
    q, k, v, do = make(2, 90, 4, 2, 32, "f16")
    off = offsets_of([50, 40])
    out, lse = lib.attention(q, k, v, offsets=off)
    grads = [host(t) for t in lib.attention_backward(do, q, k, v, out, lse, offsets=off)]
    x = [host(t) for t in (q, k, v)]
    u = [rng.standard_normal(t.shape) for t in x]
    h = 1e-5

    def f(e):
        return np.sum(host(do) * L.attention(*(a + e * b for a, b in zip(x, u)), offsets=[0, 50, 90])[0])
    slope = (f(h) - f(-h)) / (2 * h)
    got = sum(np.sum(a * b) for a, b in zip(grads, u))
    size = np.sqrt(sum(np.sum((a * b) ** 2) for a, b in zip(grads, u)))
    # every gradient is off by a few roundings of its own, independent of each other
    assert abs(got - slope) <= 6 * 4 * HALF["f16"] * size + 1e-6


def test_empty(lib):
    import torch
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    k = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = lib.attention(q, k, k)
    assert out.shape == q.shape and lse.shape == (4, 0)
    assert [t.shape for t in lib.attention_backward(q, q, k, k, out, lse)] == [q.shape, k.shape, k.shape]
    q, k, v, do = make(1, 20, 2, 2, 64, "bf16")
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 3.0)
    lib.attention(q, k, v, offsets=none, out=out)
    assert (out == 3).all()


def test_same_every_time_captured_and_on_another_stream(lib):
    import torch
    lens = [300, 1, 0, 129, 600]
    q, k, v, do = make(21, sum(lens), 8, 2, 128, "bf16")
    off = offsets_of(lens)

    def run():
        out, lse = lib.attention(q, k, v, offsets=off)
        return (out, lse) + lib.attention_backward(do, q, k, v, out, lse, offsets=off)
    want = [t.clone() for t in run()]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(run(), want))
