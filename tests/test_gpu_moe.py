"""GPU: routing, expert order and combination against the float64 oracle.

Routing is computed in 64 bits and rounded once, so ids have to be the oracle's and a
weight may be off by half a step of fp32 (2^-24 of it) plus what two 64-bit evaluations
differ by (1e-12 of the magnitudes in it). The same for its gradient, rounded to the
logits' type.
"""
import numpy as np
import pytest

from oracle import moe as R

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dt(torch, dtype))).cuda()


def host(t):
    return t.detach().cpu().double().numpy()


def make_logits(rng, T, E, dtype, masked=False):
    l = 1.5 * rng.standard_normal((T, E)).astype(np.float32)
    if masked:
        l[rng.random((T, E)) < 0.3] = -np.inf
        l[::3] = -np.inf
        l[1::4, 1:] = -np.inf
    return dev(l, dtype)


CONFIGS = [
    dict(E=1, top_k=1), dict(E=8, top_k=8), dict(E=8, top_k=2, renormalize=0, scale=2.5), dict(E=64, top_k=6),
    dict(E=64, top_k=6, score="sigmoid", bias=True, n_groups=8, top_groups=4),
    dict(E=40, top_k=3, score="sigmoid", n_groups=4, top_groups=2, group_top=1),
    dict(E=96, top_k=7, n_groups=8, top_groups=3, bias=True), dict(E=128, top_k=4, score="sigmoid", bias=True),
    dict(E=256, top_k=8, score="sigmoid", bias=True, n_groups=8, top_groups=4, scale=2.5),
    dict(E=300, top_k=32, n_groups=3, top_groups=1), dict(E=1024, top_k=32, score="sigmoid", n_groups=64, top_groups=5),
]


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cfg", CONFIGS, ids=lambda c: "-".join(f"{v}" for v in c.values()))
def test_route_and_gradient(lib, cfg, dtype, masked):
    import torch
    cfg = dict(cfg)
    E, has_bias = cfg.pop("E"), cfg.pop("bias", False)
    h = lib.route_hyper(**cfg)
    kw = dict(cfg, renormalize=bool(cfg.get("renormalize", 1)))
    K = cfg["top_k"]
    for T in (1, 5, 130):
        rng = np.random.default_rng([T, E])
        l = make_logits(rng, T, E, dtype, masked)
        bias = rng.standard_normal(E).astype(np.float32) * 0.2 if has_bias else None
        ids, w = lib.route(l, h, bias=None if bias is None else dev(bias))
        want_ids, want_w = R.route(host(l), bias=bias, **kw)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert np.all(np.abs(host(w) - want_w) <= 2.0 ** -24 * want_w + 1e-12 * cfg.get("scale", 1.0) + 2.0 ** -149)

        dw = rng.standard_normal((T, K)).astype(np.float32)
        d = lib.route_backward(dev(dw), l, ids, h)
        back = {k: kw[k] for k in ("score", "renormalize", "scale") if k in kw}
        want = R.route_backward(dw.astype(np.float64), host(l), want_ids, **back)
        mag = np.abs(dw).max() * K * cfg.get("scale", 1.0)
        got = host(d)
        tol = HALF[dtype] * np.abs(want) + 1e-11 * mag + TINY[dtype]
        assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [0, 1])
def test_route_gradient_by_differences(lib, score, renormalize):
    # central differences of the oracle's weights with the choice held fixed: for a step h
    # they are off by h^2 / 6 of the third derivative (at most 8 of the magnitudes here)
    rng = np.random.default_rng(3)
    T, E, K = 4, 12, 3
    l = rng.standard_normal((T, E)).astype(np.float32)
    h = lib.route_hyper(score=score, renormalize=renormalize, top_k=K, scale=1.5)
    ids, _ = lib.route(dev(l), h)
    dw = rng.standard_normal((T, K)).astype(np.float32)
    got = host(lib.route_backward(dev(dw), dev(l), ids, h))
    ids = ids.cpu().numpy()
    step = 1e-4

    def loss(x):
        s = R.scores(x, score)
        w = np.take_along_axis(s, ids, axis=1)
        if renormalize:
            w = w / (w.sum(axis=1, keepdims=True) + 1e-20)
        return (1.5 * w * dw).sum()

    for t in range(T):
        for e in range(E):
            up, down = l.astype(np.float64), l.astype(np.float64)
            up[t, e] += step
            down[t, e] -= step
            diff = (loss(up) - loss(down)) / (2 * step)
            mag = 1.5 * np.abs(dw[t]).sum()
            assert abs(diff - got[t, e]) <= (8 * step ** 2 + 1e-10 / step * 1e-4 + 2.0 ** -24) * mag


def test_route_ties_go_to_the_lowest_index(lib):
    import torch
    for E in (8, 70, 300):
        l = torch.zeros(3, E, device="cuda")
        l[1, E // 2:] = 1.0
        ids, w = lib.route(l, lib.route_hyper(top_k=4))
        assert ids[0].tolist() == [0, 1, 2, 3]
        assert ids[1].tolist() == [E // 2 + i for i in range(4)]
        assert torch.all(w == 0.25)
        ids, _ = lib.route(l[:, :E // 2 * 2], lib.route_hyper(top_k=2, n_groups=2))
        assert ids[0].tolist() == [0, 1]


def test_route_rows_without_an_expert(lib):
    # a padding token's row of -inf chooses none, weighs nothing and has no gradient; the
    # lowest finite logits are a choice like any other
    import torch
    l = torch.full((4, 16), -float("inf"), device="cuda")
    l[1, 3] = 0.5
    l[2] = torch.finfo(torch.float32).min
    l[3, 5], l[3, 9] = -1e30, 2.0
    for score in ("softmax", "sigmoid"):
        h = lib.route_hyper(top_k=3, score=score)
        ids, w = lib.route(l, h)
        assert ids.tolist() == [[-1, -1, -1], [3, -1, -1], [0, 1, 2], [9, 5, -1]]
        assert torch.all(w[0] == 0) and w[1].tolist() == [1.0, 0.0, 0.0]
        d = lib.route_backward(torch.ones_like(w), l, ids, h)
        assert torch.all(torch.isfinite(d)) and torch.all(d[0] == 0)
    bias = torch.zeros(16, device="cuda")
    bias[3] = -float("inf")       # a bias of -inf takes an expert out
    ids, _ = lib.route(l, lib.route_hyper(top_k=3), bias=bias)
    assert ids[1].tolist() == [-1, -1, -1] and 3 not in ids[2].tolist()


def test_route_nan_and_infinity(lib):
    # ids stay valid and distinct; a softmax over a NaN or +inf has NaN weights, other rows
    # are untouched
    import torch
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 40)).astype(np.float32)
    l = dev(x)
    l[1, 7] = float("nan")
    l[2, 7] = float("inf")
    ids, w = lib.route(l, lib.route_hyper(top_k=5))
    assert torch.all((ids >= 0) & (ids < 40))
    for row in ids.tolist():
        assert len(set(row)) == 5
    assert torch.all(torch.isnan(w[1:])) and torch.all(torch.isfinite(w[0]))
    ids, w = lib.route(l, lib.route_hyper(top_k=5, score="sigmoid"))
    assert 7 not in ids[1].tolist() and ids[2, 0] == 7 and torch.all(torch.isfinite(w))


def test_route_reads_strided_logits(lib):
    import torch
    rng = np.random.default_rng(2)
    big = dev(rng.standard_normal((20, 50)).astype(np.float32), "bf16")
    v = big[::2, 3:43]
    ids, w = lib.route(v, lib.route_hyper(top_k=4))
    ids2, w2 = lib.route(v.contiguous(), lib.route_hyper(top_k=4))
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    d = torch.full((10, 60), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.route_backward(torch.ones_like(w), v, ids, lib.route_hyper(top_k=4), dlogits=d[:, 10:50])
    assert torch.all(d[:, :10] == 7) and torch.all(d[:, 50:] == 7)


@pytest.mark.parametrize("n,E,align", [(0, 4, 128), (1, 1, 1), (7, 3, 16), (1000, 64, 128), (4096, 5, 1), (4097, 8, 64),
                                       (20000, 64, 128), (30001, 1024, 7), (300000, 3, 1024)])
def test_expert_order(lib, n, E, align):
    import torch
    rng = np.random.default_rng([n, E])
    ids = rng.integers(0, E, n).astype(np.int32)
    if n > 5:
        ids[rng.random(n) < 0.1] = -1
        ids[3], ids[4] = E, 2 ** 31 - 1      # not an expert: no row
        if E > 2:
            ids[ids == 1] = 2                # an expert without slots
    cap = n + E * (align - 1) + 37
    rows = torch.full((cap,), 99, dtype=torch.int32, device="cuda")
    offsets, counts, rows, pos = lib.expert_order(dev(ids), E, align=align, rows=rows)
    want = R.expert_order(ids, E, align, cap)
    for got, w in zip((offsets, counts, rows, pos), want):
        assert np.array_equal(got.cpu().numpy(), w)
    # the order of two runs is the same one
    again = lib.expert_order(dev(ids), E, align=align, rows=torch.empty_like(rows))
    for x, y in zip((offsets, counts, rows, pos), again):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,K,cols", [(1, 1, 1), (3, 2, 7), (5, 32, 100), (40, 6, 2048), (9, 3, 2049), (2, 4, 5000)])
def test_combine_and_gradient(lib, T, K, cols, dtype):
    # positions in any order, some slots without a row. Forward: K products and sums in
    # fp32, one rounding. Gradient: a sum of `cols` terms in fp32 (at most cols + 8
    # roundings), and one product rounded in fp32 and again to the type.
    import torch
    rng = np.random.default_rng([T, K, cols])
    n_rows = T * K + 5
    o = dev(rng.standard_normal((n_rows, cols)).astype(np.float32), dtype)
    pos = rng.permutation(n_rows)[:T * K].reshape(T, K).astype(np.int32)
    pos[rng.random((T, K)) < 0.15] = -1
    if T > 2:
        pos[1] = -1
        pos[2, 0] = n_rows       # beyond the rows
    w = rng.standard_normal((T, K)).astype(np.float32)
    dy = dev(rng.standard_normal((T, cols)).astype(np.float32), dtype)
    y = host(lib.combine(o, dev(pos), dev(w)))
    want, mag = R.combine(host(o), pos, w.astype(np.float64))
    tol = 2 * K * 2.0 ** -24 * mag
    assert np.all(np.abs(y - want) <= tol + HALF[dtype] * (np.abs(want) + tol) + TINY[dtype])
    do = torch.full_like(o, 7.0)
    dw, do = lib.combine_backward(dy, o, dev(pos), dev(w), do=do)
    want_dw, mag, want_do, written = R.combine_backward(host(dy), host(o), pos, w.astype(np.float64))
    assert np.all(np.abs(host(dw) - want_dw) <= (cols + 8) * 2.0 ** -24 * mag)
    got = host(do)
    assert np.all(got[~written] == 7.0)
    half = HALF[dtype] + 2.0 ** -24
    assert np.all(np.abs(got - want_do)[written] <= half * np.abs(want_do)[written] * (1 + 2.0 ** -7) + TINY[dtype])
    dw2, do2 = lib.combine_backward(dy, o, dev(pos), dev(w))
    assert torch.equal(dw, dw2) and np.all(host(do2)[~written] == 0)


def test_combine_gradient_by_differences(lib):
    # L = <dy, combine(o, w)> is linear in every weight and every row
    rng = np.random.default_rng(4)
    o = rng.standard_normal((12, 33)).astype(np.float32)
    pos = rng.permutation(12).reshape(4, 3).astype(np.int32)
    w = rng.standard_normal((4, 3)).astype(np.float32)
    dy = rng.standard_normal((4, 33)).astype(np.float32)
    dw, do = (host(t) for t in lib.combine_backward(dev(dy), dev(o), dev(pos), dev(w)))
    loss = lambda oo, ww: (dy * R.combine(oo, pos, ww)[0]).sum()   # noqa: E731
    o, w = o.astype(np.float64), w.astype(np.float64)
    base = loss(o, w)
    mag = R.combine_backward(dy, o, pos, w)[1]
    for t in range(4):
        for j in range(3):
            w2 = w.copy()
            w2[t, j] += 1.0
            assert abs(loss(o, w2) - base - dw[t, j]) <= 41 * 2.0 ** -24 * mag[t, j] + 1e-9
    for r, c in ((0, 0), (11, 32), (5, 7)):
        o2 = o.copy()
        o2[r, c] += 1.0
        assert abs(loss(o2, w) - base - do[r, c]) <= 2.0 ** -24 * abs(do[r, c]) + 1e-9


def test_combine_views(lib):
    # rows with their own pitch, at places where 16-byte accesses do not fit
    import torch
    rng = np.random.default_rng(6)
    buf = dev(rng.standard_normal((40, 71)).astype(np.float32), "bf16")
    pos = dev(rng.permutation(40)[:24].reshape(8, 3).astype(np.int32))
    w = dev(rng.random((8, 3)).astype(np.float32))
    for lo, hi in ((0, 64), (3, 68), (7, 8)):
        y = torch.full((8, 80), 7.0, dtype=torch.bfloat16, device="cuda")
        lib.combine(buf[:, lo:hi], pos, w, out=y[:, 5:5 + hi - lo])
        assert torch.equal(y[:, 5:5 + hi - lo], lib.combine(buf[:, lo:hi].contiguous(), pos, w))
        assert torch.all(y[:, :5] == 7) and torch.all(y[:, 5 + hi - lo:] == 7)


@pytest.mark.parametrize("n,E,align", [(0, 3, 128), (96, 64, 16), (5000, 40, 128)])
def test_expert_order_allocates_its_results(lib, n, E, align):
    import torch
    ids = np.random.default_rng([n, 31]).integers(-1, E, n).astype(np.int32)
    want = R.expert_order(ids, E, align, n + E * (align - 1))
    got = lib.expert_order(dev(ids), E, align=align)
    later = lib.expert_order(dev(ids[::-1].copy()), E, align=align)   # results of their own
    assert [t.is_contiguous() and t.dtype == torch.int32 for t in got] == [True] * 4
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert not {t.data_ptr() for t in got if t.numel()} & {t.data_ptr() for t in later if t.numel()}


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top_groups,K", [(64, 1, 1, 6), (64, 32, 7, 6), (64, 64, 9, 6), (33, 33, 4, 4),
                                                   (33, 1, 1, 32), (32, 8, 2, 5), (63, 21, 3, 5)])
def test_route_rows_do_not_meet_their_neighbours(lib, E, groups, top_groups, K, score):
    # neighbouring rows share a wave: rows of ties, of no expert, of few experts and of NaN
    # next to ordinary ones, in every pairing
    rng = np.random.default_rng([E, groups])
    kinds = [(a, b) for a in range(5) for b in range(5)]
    l = rng.standard_normal((2 * len(kinds) + 1, E)).astype(np.float32)
    for i, kind in enumerate(k for pair in kinds for k in pair):
        if kind == 1:
            l[i] = 0.5                                   # ties
        elif kind == 2:
            l[i] = -np.inf                               # no expert
        elif kind == 3:
            l[i, rng.permutation(E)[: E - 3]] = -np.inf  # three experts
        elif kind == 4:
            l[i, rng.integers(E)] = np.nan
    h = lib.route_hyper(score=score, top_k=K, n_groups=groups, top_groups=top_groups)
    ids, w = lib.route(dev(l), h)
    want_ids, want_w = R.route(l.astype(np.float64), score=score, top_k=K, n_groups=groups, top_groups=top_groups)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    got = host(w)
    assert np.array_equal(np.isnan(got), np.isnan(want_w))
    ok = ~np.isnan(want_w)
    assert np.all(np.abs(got - want_w)[ok] <= (2.0 ** -24 * want_w + 1e-12)[ok])
