"""GPU: norm, embedding and clipping against the float64 oracle.

Tolerances count roundings: half a step of the output's type (HALF), and 2^-24 of the
magnitudes for each fp32 operation on the longest path to a value.
"""
import numpy as np
import pytest

from oracle import layer as L

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}
U = 2.0 ** -24
TYPES = ["f32", "bf16", "f16"]


def dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def dev(x, dtype="f32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x)).to(dt(dtype)).cuda()


def host(t):
    return t.detach().cpu().double().numpy()


def strided(x, pad, shift=0):
    """The same values in rows `pad` elements further apart, `shift` elements off an aligned
    start; what lies between is NaN."""
    import torch
    rows, cols = x.shape
    base = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=x.dtype, device=x.device)
    view = base[shift:].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    return view


def close(got, want, tol):
    err = np.abs(got - want)
    assert np.all(err <= tol), f"{np.max(err / np.maximum(tol, 1e-300)):.3f} of the tolerance at {np.argmax(err / np.maximum(tol, 1e-300))}"


# ----------------------------------------------------------------------------- norm

# fp32 operations on the way to a sum over a row: at most 32 in a lane, 6 steps across the
# wave, 8 across waves
ROW_SUM = 48


def sum_of(got, x, r, dtype):
    """The stored sum of x and r is one fp32 addition and one rounding off."""
    exact = x + r
    close(got, exact, (HALF[dtype] + 2 * U) * np.abs(exact) + TINY[dtype])


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (5, 64), (2, 127), (9, 129), (130, 512), (4, 513), (5, 1024),
                                       (6, 2047), (33, 2048), (3, 2049), (7, 4096), (2, 8191), (3, 8192), (2, 11008),
                                       (2, 16383), (3, 16384), (6, 8), (9, 1536), (5, 1531), (4, 4097), (3, 6144), (2, 6137),
                                       (3, 8193), (2, 12288), (2, 12287)])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm(lib, rows, cols, dtype):
    import torch
    rng = np.random.default_rng([rows, cols])
    x, r = dev(rng.standard_normal((rows, cols)) * 3, dtype), dev(rng.standard_normal((rows, cols)), dtype)
    for wt, residual, eps in (("f32", True, 1e-6), (dtype, False, 1e-3), (None, True, 0.0)):
        w = None if wt is None else dev(1 + 0.3 * rng.standard_normal(cols), wt)
        n = lib.rms_norm(x, w, residual=r if residual else None, eps=eps, fp8="both", fmt="e4m3")
        if residual:
            sum_of(host(n.sum), host(x), host(r), dtype)
        else:
            assert n.sum is x
        y, rstd = L.rms_norm(host(n.sum), None if w is None else host(w), eps)
        # half the relative error of the sum, then a division, a square root and a reciprocal
        close(host(n.rstd), rstd, (ROW_SUM / 2 + 6) * U * rstd)
        close(host(n.y), y, (HALF[dtype] + (ROW_SUM / 2 + 9) * U) * np.abs(y) + TINY[dtype])
        # in 8 bits: the bytes that quantising y gives
        for fmt in ("e4m3", "e5m2"):
            q = lib.fp8_quantize(n.y, fmt)
            m = lib.rms_norm(x, w, residual=r if residual else None, eps=eps, fp8="only", fmt=fmt)
            assert m.y is None and torch.equal(m.rstd, n.rstd)
            assert torch.equal(m.fp8.data.view(torch.uint8), q.data.view(torch.uint8))
            assert torch.equal(m.fp8.scale.view(torch.uint8), q.scale.view(torch.uint8))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 300), (5, 64), (4, 129), (130, 512), (7, 1000), (3500, 1536),
                                       (65, 2048), (5, 2049), (900, 4096), (3, 8191), (2, 16384), (3, 7), (6, 8), (9, 1536),
                                       (900, 1531), (4, 4097), (3, 6144), (800, 6137), (3, 8193), (2, 12288), (2, 12287)])
@pytest.mark.parametrize("dtype", TYPES)
def test_norm_gradient(lib, rows, cols, dtype):
    rng = np.random.default_rng([rows, cols, 1])
    s, dy, ds = (dev(rng.standard_normal((rows, cols)) * k, dtype) for k in (2.0, 0.1, 0.05))
    for wt, dsum, ot in (("f32", ds, "f32"), (dtype, None, dtype), (None, ds, None)):
        w = None if wt is None else dev(1 + 0.3 * rng.standard_normal(cols), wt)
        rstd = dev(L.rms_norm(host(s))[1])
        given = None if ot is None else dev(rng.standard_normal(cols), ot)
        before = None if ot is None else host(given)
        dx, dw = lib.rms_norm_backward(dy, s, w, rstd, dsum=dsum, dweight=given, accumulate=given is not None)
        hw = None if w is None else host(w)
        want, want_w = L.rms_norm_backward(host(dy), host(s), hw, host(rstd), None if dsum is None else host(dsum))
        n = np.abs(host(s)) * host(rstd)[:, None]
        g = np.abs(host(dy)) * (1.0 if hw is None else np.abs(hw))
        parts = host(rstd)[:, None] * (g + n * np.mean(g * n, axis=1, keepdims=True)) + (0 if dsum is None else np.abs(host(ds)))
        close(host(dx), want, HALF[dtype] * np.abs(want) + (ROW_SUM + 10) * U * parts + TINY[dtype])
        if w is None:
            assert dw is None
            continue
        assert dw is given
        # the longest path: a team's rows in turn, the teams, the workgroups
        steps = 4 + -(-rows // 768) + 4 + 768 / 16 + 16
        mag = np.sum(np.abs(host(dy)) * n, axis=0)
        close(host(dw), before + want_w, HALF[ot] * np.abs(before + want_w) + steps * U * (mag + np.abs(before)) + TINY[ot])
        fresh = lib.rms_norm_backward(dy, s, w, rstd, dsum=dsum)[1]
        close(host(fresh), want_w, (steps + 1) * U * mag)


def test_norm_gradient_against_differences(lib):
    rng = np.random.default_rng(5)
    rows, cols, eps = 6, 200, 1e-2
    x, w, dy, ds = rng.standard_normal((rows, cols)), 1 + 0.2 * rng.standard_normal(cols), rng.standard_normal((rows, cols)), rng.standard_normal((rows, cols))
    tx, tw, tdy, tds = dev(x), dev(w), dev(dy), dev(ds)
    x, w, dy, ds = (host(t) for t in (tx, tw, tdy, tds))
    n = lib.rms_norm(tx, tw, eps=eps)
    dx, dw = lib.rms_norm_backward(tdy, tx, tw, n.rstd, dsum=tds)
    ux, uw = rng.standard_normal((rows, cols)), rng.standard_normal(cols)

    def f(h):
        return np.sum(dy * L.rms_norm(x + h * ux, w + h * uw, eps)[0]) + np.sum(ds * (x + h * ux))
    h = 1e-5
    slope = (f(h) - f(-h)) / (2 * h)
    got = np.sum(host(dx) * ux) + np.sum(host(dw) * uw)
    scale = np.sum(np.abs(host(dx) * ux)) + np.sum(np.abs(host(dw) * uw))
    assert abs(got - slope) <= (2 * ROW_SUM * U + 1e-8) * scale   # differences in 64 bits: h^2 and 1e-16 / h


@pytest.mark.parametrize("dtype", TYPES)
def test_norm_strides_and_neighbours(lib, dtype):
    import torch
    rng = np.random.default_rng(7)
    for rows, cols, pad, shift in ((5, 100, 3, 1), (9, 1000, 8, 3), (4, 3000, 1, 5)):
        x, r, dy = (dev(rng.standard_normal((rows, cols)), dtype) for _ in range(3))
        w = dev(1 + 0.3 * rng.standard_normal(cols), dtype)
        want = lib.rms_norm(x, w, residual=r)
        sx, sr = strided(x, pad, shift), strided(r, pad + 2, shift)
        out, total = strided(x, pad, shift), strided(x, pad + 1, shift)
        got = lib.rms_norm(sx, w, residual=sr, out=out, out_sum=total)
        assert got.y is out and got.sum is total
        assert torch.equal(got.y, want.y) and torch.equal(got.sum, want.sum) and torch.equal(got.rstd, want.rstd)
        for view, p in ((out, pad), (total, pad + 1)):   # what lies between the rows stays
            between = view.as_strided((rows - 1, p), view.stride(), view.storage_offset() + cols)
            assert torch.isnan(between).all()
        dx, dw = lib.rms_norm_backward(dy, want.sum, w, want.rstd, dsum=r)
        gx, gw = lib.rms_norm_backward(strided(dy, pad, shift), got.sum, w, want.rstd, dsum=sr, dx=out)
        assert gx is out and torch.equal(gx, dx) and torch.equal(gw, dw)
        wide = x[:1].expand(rows, cols)   # one row for all
        assert torch.equal(lib.rms_norm(wide, w).y, lib.rms_norm(wide.contiguous(), w).y)


def test_norm_values_that_are_not_finite_stay_in_their_row(lib):
    import torch
    x = torch.randn(6, 700, device="cuda").to(torch.bfloat16)
    want = lib.rms_norm(x, fp8="both")
    y = x.clone()
    y[1, 3], y[4, 600] = float("inf"), float("nan")
    y[2] = 0
    got = lib.rms_norm(y, fp8="both")
    keep = [0, 3, 5]
    assert torch.equal(got.y[keep], want.y[keep]) and torch.equal(got.rstd[keep], want.rstd[keep])
    assert torch.equal(got.fp8.data.view(torch.uint8)[keep], want.fp8.data.view(torch.uint8)[keep])
    assert torch.isnan(got.y[4]).all() and torch.isnan(got.y[1, 3]) and (got.y[1, :3] == 0).all() and (got.y[2] == 0).all()


def test_norm_of_no_rows(lib):
    import torch
    x, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    n = lib.rms_norm(x, w, fp8="both")
    assert n.y.shape == (0, 64) and n.rstd.shape == (0,)
    dw = torch.full((64,), 3.0, device="cuda")
    assert (lib.rms_norm_backward(x, x, w, n.rstd)[1] == 0).all()
    lib.rms_norm_backward(x, x, w, n.rstd, dweight=dw, accumulate=True)
    assert (dw == 3).all()


# ----------------------------------------------------------------------------- embedding

def make_ids(rng, tokens, vocab, kind):
    if kind == "one":
        ids = np.full(tokens, vocab - 1)
    elif kind == "hot":   # a few ids take most of the tokens
        ids = np.where(rng.random(tokens) < 0.7, rng.integers(0, 2, tokens) * (vocab - 1), rng.integers(0, vocab, tokens))
    else:
        ids = rng.integers(0, vocab, tokens)
    bad = rng.random(tokens) < 0.1
    if kind == "mixed":
        ids = np.where(bad, rng.choice([-1, -7, vocab, vocab + 5, -2 ** 31, 2 ** 31 - 1], tokens), ids)
    elif kind == "none":
        ids = np.full(tokens, -1)
    return ids


@pytest.mark.parametrize("tokens,vocab,cols", [(1, 1, 1), (7, 3, 9), (33, 1, 40), (64, 255, 8), (65, 256, 512), (100, 300, 513),
                                               (1000, 70000, 65), (4096, 32000, 130), (4097, 1000, 2049), (9000, 511, 96),
                                               (16384, 40, 24), (4097, 300, 520), (8192, 3000, 40), (8193, 3000, 40)])
@pytest.mark.parametrize("kind", ["even", "hot", "one", "mixed", "none"])
def test_embedding_and_gradient(lib, tokens, vocab, cols, kind):
    import torch
    rng = np.random.default_rng([tokens, vocab, cols])
    ids = make_ids(rng, tokens, vocab, kind)
    combos = [("f32", "bf16", "f32", 1.0), ("bf16", "bf16", "bf16", 8.0), ("f16", "f16", "f32", 0.3), ("f32", "f32", "f16", 1.7)]
    for k, (tt, yt, gt, scale) in enumerate(combos[:2 if tokens * cols > 10 ** 5 else 4]):
        tid = torch.from_numpy(ids.astype(np.int64 if k % 2 else np.int32)).cuda()
        table, dy = dev(rng.standard_normal((vocab, cols)), tt), dev(rng.standard_normal((tokens, cols)), yt)
        s32 = float(np.float32(scale))
        y = lib.embedding(tid, table, scale=scale, out_dtype=dt(yt))
        want = L.embedding(ids, host(table), s32)
        close(host(y), want, (HALF[yt] + U) * np.abs(want) + TINY[yt])
        g = lib.embedding_backward(dy, tid, vocab, scale=scale, out_dtype=dt(gt))
        want, mag, count = L.embedding_backward(host(dy), ids, vocab, s32)
        # a chunk's tokens in turn (8 or 32), then the chunks, the product and the sum with what is there
        steps = np.maximum(np.minimum(count, 32) + np.ceil(count / 32), np.minimum(count, 8) + np.ceil(count / 8)) + 4
        tol = HALF[gt] * np.abs(want) + steps[:, None] * U * mag + TINY[gt]
        close(host(g), want, tol)
        assert torch.equal(g, lib.embedding_backward(dy, tid, vocab, scale=scale, out_dtype=dt(gt)))
        before = dev(rng.standard_normal((vocab, cols)), gt)
        old = host(before)
        got = lib.embedding_backward(dy, tid, vocab, scale=scale, out=before, accumulate=True)
        assert got is before
        close(host(got), old + want, HALF[gt] * np.abs(old + want) + steps[:, None] * U * (mag + np.abs(old)) + TINY[gt])
        assert np.array_equal(host(got)[count == 0], old[count == 0])


def test_embedding_strides_shapes_and_empty(lib):
    import torch
    rng = np.random.default_rng(3)
    table = dev(rng.standard_normal((50, 37)), "bf16")
    ids = torch.from_numpy(rng.integers(-1, 50, (4, 9))).cuda()
    y = lib.embedding(ids, table)
    assert y.shape == (4, 9, 37) and torch.equal(y, lib.embedding(ids, strided(table, 5, 1)))
    dy = torch.randn(4, 9, 37, device="cuda")
    g = lib.embedding_backward(dy, ids, 50)
    packed = strided(torch.zeros(50, 37, device="cuda"), 3, 1)
    got = lib.embedding_backward(strided(dy.view(36, 37), 4, 3), ids.view(-1), 50, out=packed)
    assert got is packed and torch.equal(got, g)
    assert torch.isnan(packed.as_strided((49, 3), packed.stride(), packed.storage_offset() + 37)).all()
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert lib.embedding(none, table).shape == (0, 37)
    assert (lib.embedding_backward(torch.empty(0, 37, device="cuda"), none, 50) == 0).all()
    assert torch.equal(lib.embedding_backward(torch.empty(0, 37, device="cuda"), none, 50, out=g.clone(), accumulate=True), g)


def test_embedding_gradient_against_differences(lib):
    rng = np.random.default_rng(11)
    import torch
    ids = rng.integers(-1, 20, 300)
    dy, u = dev(rng.standard_normal((300, 33))), rng.standard_normal((20, 33))
    g = lib.embedding_backward(dy, torch.from_numpy(ids).cuda(), 20, scale=2.0)
    # linear in the table: the difference is exact for any step
    slope = np.sum(host(dy) * L.embedding(ids, u, 2.0))
    assert abs(np.sum(host(g) * u) - slope) <= 64 * U * np.sum(np.abs(host(dy) * L.embedding(ids, u, 2.0)))


def test_embedding_no_value_of_another_row(lib):
    """A token's NaN reaches its own row alone, and a NaN row only the tokens that ask for it."""
    import torch
    ids = torch.arange(200, device="cuda") % 50
    dy = torch.randn(200, 600, device="cuda")
    want = lib.embedding_backward(dy, ids, 60)
    dy[57] = float("nan")
    got = lib.embedding_backward(dy, ids, 60)
    assert torch.isnan(got[7]).all()
    keep = [i for i in range(60) if i != 7]
    assert torch.equal(got[keep], want[keep])


# ----------------------------------------------------------------------------- clipping

def make_grads(rng, sizes, types, scale=1.0):
    import torch
    return [dev(rng.standard_normal(n) * scale, t) if n else torch.empty(0, dtype=dt(t), device="cuda")
            for n, t in zip(sizes, types)]


SIZES = [[1], [5, 0, 8191], [8192, 8193, 3], [70001], [17] * 119 + [9000], list(range(1, 260)), [0, 0]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_clip(lib, sizes):
    import torch
    rng = np.random.default_rng(len(sizes))
    for mix in (["f32"], ["bf16"], ["f16"], ["bf16", "f32", "f16"]):
        types = [mix[i % len(mix)] for i in range(len(sizes))]
        grads = make_grads(rng, sizes, types)
        values = [host(g) for g in grads]
        exact = sum(float(np.sum(v * v)) for v in values)
        sumsq = lib.grad_sumsq(grads)
        assert sumsq.dtype == torch.float64 and sumsq.shape == ()
        assert abs(sumsq.item() - exact) <= 1e-13 * exact
        assert lib.grad_sumsq(grads, out=sumsq.clone(), accumulate=True).item() == 2 * sumsq.item()
        for share in (0.3, 5.0):
            max_norm = share * np.sqrt(exact)
            norm, want = L.clip(values, float(np.float32(max_norm)))
            for ot in ("f32", "bf16", "f16", None):
                outs = [torch.full_like(g, float("nan"), dtype=dt(ot)) for g in grads] if ot else None
                ins = grads if ot else [g.clone() for g in grads]
                got = lib.clip_gradients(ins, max_norm, out=outs)
                assert got.shape == () and abs(got.item() - norm) <= 2 * U * norm
                for o, w, t in zip(outs or ins, want, types):
                    close(host(o), w, (HALF[ot or t] + 3 * U) * np.abs(w) + TINY[ot or t])
                if share > 1 and not ot:
                    assert all(torch.equal(i, g) for i, g in zip(ins, grads))


def test_clip_far_values(lib):
    """Squares far outside the range of 32 bits, and sums that mix them."""
    import torch
    for scale in (1e30, 1e-30):
        g = [torch.full((10000,), scale, device="cuda"), torch.full((77,), -scale, device="cuda")]
        norm = lib.clip_gradients(g, scale)
        assert abs(norm.item() / (scale * np.sqrt(10077)) - 1) <= 4 * U
        if scale > 1:
            want = scale / np.sqrt(10077)
            assert torch.all((g[0] / want - 1).abs() <= 8 * U)
    # the smallest norms: 1e-6 is added to them, as the formula has it
    assert (g[0] == torch.tensor(1e-30 * min(1.0, 1e-30 / 1e-6), device="cuda")).all()


def test_clip_norms_that_are_not_finite(lib):
    import torch
    g = torch.ones(5000, device="cuda")
    g[77] = float("inf")
    h = [g, torch.ones(3, device="cuda")]
    assert lib.clip_gradients(h, 1.0).item() == float("inf")
    assert torch.isnan(h[0][77]) and (h[0][:77] == 0).all() and (h[1] == 0).all()
    h = [torch.full((9,), float("nan"), device="cuda"), torch.ones(3, device="cuda")]
    assert np.isnan(lib.clip_gradients(h, 1.0).item()) and torch.isnan(h[1]).all()


def test_clip_without_limit(lib):
    """An infinite max_norm leaves every value as it is, and still gives the norm; zero leaves zeros."""
    import torch
    for bad in (3.0, float("inf"), float("nan")):
        g = torch.ones(5000, device="cuda")
        g[77] = bad
        out = torch.zeros(5000, device="cuda")
        assert np.array_equal(lib.clip_gradients([g], float("inf"), out=[out]).item(), np.sqrt(host(g).__pow__(2).sum()).astype(np.float32),
                              equal_nan=True)
        assert np.array_equal(host(out), host(g), equal_nan=True)
    g = torch.ones(5000, device="cuda")
    lib.clip_gradients([g], 0.0)
    assert (g == 0).all()


def test_clip_into_the_packed_gradients_and_by_shards(lib):
    import torch
    rng = np.random.default_rng(2)
    a, b = dev(rng.standard_normal((64, 48))), dev(rng.standard_normal((40, 64)))
    packed = torch.full((64 * 48 + 64 + 40 * 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    views = [packed[:64 * 48].view(64, 48), packed[64 * 48 + 64:].view(40, 64)]
    total = lib.grad_sumsq([a]) + lib.grad_sumsq([b])     # as two ranks add them up
    norm = lib.clip_gradients([a, b], 2.0, sumsq=total, out=views)
    want = L.clip([host(a), host(b)], 2.0)
    assert abs(norm.item() - want[0]) <= 2 * U * want[0]
    for v, w in zip(views, want[1]):
        close(host(v), w, (HALF["bf16"] + 3 * U) * np.abs(w))
    assert (packed[64 * 48:64 * 48 + 64] == 7).all()


# ----------------------------------------------------------------------------- far offsets

def test_elements_beyond_2_31(lib):
    import torch
    rows, ld = 40, 1 << 26   # 5.4 GB of bf16
    base, other, third = (torch.empty(rows * ld, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    x = torch.randn(rows, 300, device="cuda").bfloat16()
    view = base.as_strided((rows, 300), (ld, 1), 8)
    view.copy_(x)
    out = other.as_strided((rows, 300), (ld, 1), 4096)
    want = lib.rms_norm(x)
    assert torch.equal(lib.rms_norm(view, out=out).y, want.y)
    dx = third.as_strided((rows, 300), (ld, 1), 8192)
    assert torch.equal(lib.rms_norm_backward(out, view, None, want.rstd, dx=dx)[0],
                       lib.rms_norm_backward(want.y, x, None, want.rstd)[0])
    ids = torch.randint(0, rows, (500,), device="cuda")
    assert torch.equal(lib.embedding(ids, view), lib.embedding(ids, x))
    dy = torch.randn(500, 300, device="cuda").bfloat16()
    table = third.as_strided((rows, 300), (ld, 1), 12288)
    assert torch.equal(lib.embedding_backward(dy, ids, rows, out=table), lib.embedding_backward(dy, ids, rows, out_dtype=torch.bfloat16))
    base.zero_()
    base[::1 << 20] = 2.0   # 2560 of 2.7e9 elements
    n = base[::1 << 20].numel()
    norm = lib.clip_gradients([base[:-3]], 1.0)
    assert norm.item() == np.float32(2.0 * np.sqrt(n))
    assert torch.equal(base[::1 << 20], torch.full((n,), 2.0, device="cuda").mul_(1.0 / norm.double()).bfloat16())


# ----------------------------------------------------------------------------- streams, graphs

def operators(lib):
    """Calls of every operator on fixed inputs: name -> function that returns its outputs."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)

    def n(*s):
        return torch.randn(*s, generator=g, device="cuda")
    x, r, dy = n(300, 1500).bfloat16(), n(300, 1500).bfloat16(), n(300, 1500).bfloat16()
    w = n(1500)
    table, ids = n(700, 130), torch.randint(-1, 700, (6000,), generator=g, device="cuda")
    de = n(6000, 130).bfloat16()
    grads = [n(9000), n(77), n(40000)]
    rstd = lib.rms_norm(x, w).rstd

    def norm():
        o = lib.rms_norm(x, w, residual=r, fp8="both")
        return o.y, o.sum, o.rstd, o.fp8.data.view(torch.uint8), o.fp8.scale.view(torch.uint8)

    def clip():
        outs = [torch.empty_like(t) for t in grads]
        return [lib.clip_gradients(grads, 3.0, out=outs)] + outs
    q, k = n(500, 8, 64).bfloat16(), n(500, 2, 64).bfloat16()
    off = torch.tensor([0, 120, 500], dtype=torch.int32, device="cuda")
    o, lse = lib.attention(q, k, k, offsets=off)
    return {"attention": lambda: lib.attention(q, k, k, offsets=off),
            "attention gradient": lambda: lib.attention_backward(o, q, k, k, o, lse, offsets=off),
            "norm": norm, "norm gradient": lambda: lib.rms_norm_backward(dy, x, w, rstd, dsum=r),
            "embedding": lambda: [lib.embedding(ids, table, scale=2.0)],
            "embedding gradient": lambda: [lib.embedding_backward(de, ids, 700)], "clip": clip}


def test_three_threads_at_once(lib):
    """Threads on one stream and on streams of their own: no call sees another one's workspace."""
    import threading

    import torch
    runs = operators(lib)
    want = {n: [t.clone() for t in f()] for n, f in runs.items()}
    torch.cuda.synchronize()
    bad = []

    def work(own):
        stream = torch.cuda.Stream() if own else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                for n, f in runs.items():
                    got = f()
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[n])):
                        bad.append(n)
    threads = [threading.Thread(target=work, args=(i == 2,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


NAMES = ["norm", "norm gradient", "embedding", "embedding gradient", "clip", "attention", "attention gradient"]


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_on_another_stream(lib, name):
    import torch
    run = operators(lib)[name]
    want = [t.clone() for t in run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for k in range(3):
        for t in got:
            t.view(-1)[:1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(run(), want))   # eager work in between
