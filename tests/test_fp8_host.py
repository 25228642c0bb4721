"""The 8-bit and mixture-of-experts entry points without a GPU: every refusal, before
any device work (the addresses are never dereferenced), the operand layout, and the
oracle's own values."""
import ctypes

import numpy as np
import pytest

import newton_schulz_step_amd as nss
from newton_schulz_step_amd import _binding as B
from oracle import fp8 as F
from oracle import moe as R

FAKE = 0x7f0000000000
GIB = 1 << 30


def at(i):
    return FAKE + i * 64 * GIB


@pytest.fixture(scope="module")
def lib():
    return nss.load()


def operand(i, rows=40, cols=300, batch=1, fmt=0, **kw):
    f = dict(data=at(i), scale=at(i) + 32 * GIB, batch=batch, rows=rows, cols=cols, format=fmt)
    f.update(kw)
    return B.Fp8Operand(f["data"], f["scale"], f["batch"], f["rows"], f["cols"], f["format"], 0)


def source(rows=40, cols=300, **kw):
    f = dict(data=at(0), batch_stride=0, ld=cols, batch=1, rows=rows, cols=cols, dtype=1, row_div=1, row_index=None,
             out_rows=rows, row_weight=None, n_weights=0)
    f.update(kw)
    return B.Fp8Source(*[f[n] for n, _ in B.Fp8Source._fields_])


def ref(x):
    return None if x is None else ctypes.byref(x)


def quantize(lib, src, out=None, out_t=None, blocks=0):
    return lib.muon_fp8_quantize(ref(src), blocks, ref(out), ref(out_t), None)


def test_quantize_refusals(lib):
    q, t = operand(1), operand(2, 300, 40)
    ok = source()
    assert quantize(lib, None, q) == nss.ERR_NULL
    assert quantize(lib, ok) == nss.ERR_NULL
    assert quantize(lib, source(data=None), q) == nss.ERR_NULL
    assert quantize(lib, ok, operand(1, data=None)) == nss.ERR_NULL
    assert quantize(lib, ok, operand(1, scale=None)) == nss.ERR_NULL
    for bad in (operand(1, rows=41), operand(1, cols=301), operand(1, batch=2), operand(1, batch=0),
                operand(1, rows=-1), operand(1, cols=(1 << 23) + 1)):
        assert quantize(lib, ok, bad) == nss.ERR_BAD_SHAPE
    assert quantize(lib, ok, None, operand(2, 40, 300)) == nss.ERR_BAD_SHAPE
    assert quantize(lib, ok, q, operand(2, 300, 40, fmt=1)) == nss.ERR_UNSUPPORTED
    assert quantize(lib, ok, operand(1, fmt=2)) == nss.ERR_UNSUPPORTED
    assert quantize(lib, source(dtype=3), q) == nss.ERR_UNSUPPORTED
    assert quantize(lib, source(rows=-1, out_rows=-1), q) == nss.ERR_BAD_SHAPE
    assert quantize(lib, source(batch=1025), q) == nss.ERR_BAD_SHAPE
    assert quantize(lib, source(ld=-1), q) == nss.ERR_BAD_SHAPE
    assert quantize(lib, source(ld=1 << 29), q) == nss.ERR_BAD_SHAPE
    assert quantize(lib, source(out_rows=41), operand(1, rows=41)) == nss.ERR_BAD_SHAPE
    assert quantize(lib, source(row_div=2), q) == nss.ERR_UNSUPPORTED
    assert quantize(lib, source(row_weight=at(5)), q) == nss.ERR_UNSUPPORTED
    assert quantize(lib, source(row_index=at(5), row_div=0), q) == nss.ERR_BAD_SHAPE
    assert quantize(lib, source(row_index=at(5), batch=2), operand(1, batch=2)) == nss.ERR_BAD_SHAPE
    assert quantize(lib, source(row_index=at(5) + 2), q) == nss.ERR_ALIGN
    assert quantize(lib, source(row_index=at(5), row_weight=at(6), n_weights=-1), q) == nss.ERR_BAD_SHAPE
    assert quantize(lib, source(data=at(0) + 1), q) == nss.ERR_ALIGN
    assert quantize(lib, ok, operand(1, data=at(1) + 8)) == nss.ERR_ALIGN
    assert quantize(lib, ok, operand(1, scale=at(3) + 2)) == nss.ERR_ALIGN
    assert quantize(lib, ok, operand(1, data=at(0) + 16 * 600)) == nss.ERR_OVERLAP      # inside the source
    assert quantize(lib, ok, operand(1, scale=at(1) + 64)) == nss.ERR_OVERLAP
    assert quantize(lib, ok, q, operand(2, 300, 40, data=at(1) + 128)) == nss.ERR_OVERLAP
    assert "out" in lib.muon_last_error().decode()
    assert quantize(lib, source(rows=0, out_rows=0, data=None), operand(1, rows=0, data=None, scale=None)) == nss.OK
    assert quantize(lib, source(cols=0), operand(1, cols=0)) == nss.OK


def matmul(lib, a, b, off=None, c=True, **kw):
    f = dict(data=at(8), batch_stride=0, ld=b.rows if b else 1, dtype=1, accumulate=0)
    f.update(kw)
    r = B.Fp8Result(f["data"], f["batch_stride"], f["ld"], f["dtype"], f["accumulate"])
    return lib.muon_fp8_matmul(ref(a), ref(b), off, ref(r) if c else None, None)


def test_matmul_refusals(lib):
    a, b = operand(1, 40, 300), operand(2, 50, 300)
    assert matmul(lib, None, b) == nss.ERR_NULL
    assert matmul(lib, a, None) == nss.ERR_NULL
    assert matmul(lib, a, b, c=False) == nss.ERR_NULL
    assert matmul(lib, a, b, data=None) == nss.ERR_NULL
    assert matmul(lib, operand(1, 40, 300, data=None), b) == nss.ERR_NULL
    assert matmul(lib, operand(1, 40, 301), b) == nss.ERR_BAD_SHAPE
    assert matmul(lib, operand(1, 40, 300, batch=2), b) == nss.ERR_BAD_SHAPE
    assert matmul(lib, a, operand(2, 50, 300, batch=1025)) == nss.ERR_BAD_SHAPE
    assert matmul(lib, a, b, ld=49) == nss.ERR_BAD_SHAPE
    assert matmul(lib, operand(1, batch=2), operand(2, 50, 300, batch=2), batch_stride=1999) == nss.ERR_BAD_SHAPE
    assert matmul(lib, a, b, dtype=3) == nss.ERR_UNSUPPORTED
    assert matmul(lib, operand(1, fmt=5), b) == nss.ERR_UNSUPPORTED
    assert matmul(lib, a, b, data=at(8) + 1) == nss.ERR_ALIGN
    assert matmul(lib, operand(1, data=at(1) + 4), b) == nss.ERR_ALIGN
    assert matmul(lib, a, b, data=at(2) + 256) == nss.ERR_OVERLAP
    assert matmul(lib, a, b, data=at(1) + 32 * GIB) == nss.ERR_OVERLAP
    # grouped: one matrix a, offsets aligned and apart from the result
    assert matmul(lib, operand(1, batch=3), operand(2, 50, 300, batch=3), off=at(9)) == nss.ERR_BAD_SHAPE
    assert matmul(lib, a, operand(2, 50, 300, batch=3), off=at(9) + 1) == nss.ERR_ALIGN
    assert matmul(lib, a, operand(2, 50, 300, batch=3), off=at(8) + 64) == nss.ERR_OVERLAP
    assert matmul(lib, operand(1, rows=0), b) == nss.OK
    assert matmul(lib, a, operand(2, rows=0)) == nss.OK


def test_matmul_grouped_k_refusals(lib):
    a, b = operand(1, 40, 384), operand(2, 50, 384)

    def run(a, b, off=at(9), n=3, c=True, **kw):
        f = dict(data=at(8), batch_stride=2000, ld=50, dtype=0, accumulate=0)
        f.update(kw)
        r = B.Fp8Result(f["data"], f["batch_stride"], f["ld"], f["dtype"], f["accumulate"])
        return lib.muon_fp8_matmul_grouped_k(ref(a), ref(b), off, n, ref(r) if c else None, None)
    assert run(a, b, off=None) == nss.ERR_NULL
    assert run(a, b, c=False) == nss.ERR_NULL
    assert run(a, b, data=None) == nss.ERR_NULL
    assert run(operand(1, 40, 384, batch=2), b) == nss.ERR_BAD_SHAPE
    assert run(a, operand(2, 50, 256)) == nss.ERR_BAD_SHAPE
    assert run(a, b, n=-1) == nss.ERR_BAD_SHAPE
    assert run(a, b, n=1025) == nss.ERR_BAD_SHAPE
    assert run(a, b, batch_stride=1999) == nss.ERR_BAD_SHAPE
    assert run(a, b, off=at(9) + 2) == nss.ERR_ALIGN
    assert run(a, b, dtype=7) == nss.ERR_UNSUPPORTED
    assert run(a, b, off=at(8)) == nss.ERR_OVERLAP
    assert run(a, b, n=0) == nss.OK


def route(lib, h, tokens=10, experts=16, logits=at(0), ids=at(1), w=at(2), bias=None, dtype=0, ld=None):
    return lib.muon_route(logits, dtype, tokens, experts, experts if ld is None else ld, bias, ref(h), ids, w, None)


def test_route_refusals(lib):
    H = nss.route_hyper
    h = H(top_k=4)
    assert route(lib, None) == nss.ERR_NULL
    for name in ("logits", "ids", "w"):
        assert route(lib, h, **{name: None}) == nss.ERR_NULL
        assert route(lib, h, **{name: at(7) + 1}) == nss.ERR_ALIGN
    assert route(lib, h, bias=at(5) + 2) == nss.ERR_ALIGN
    assert route(lib, H(top_k=4, score="tanh")) == nss.ERR_BAD_METHOD
    assert route(lib, H(top_k=4, scale=float("inf"))) == nss.ERR_BAD_HYPER
    assert route(lib, h, dtype=9) == nss.ERR_UNSUPPORTED
    for bad in (H(top_k=0), H(top_k=17), H(top_k=33), H(top_k=4, n_groups=3), H(top_k=4, n_groups=0),
                H(top_k=4, n_groups=4, top_groups=5), H(top_k=4, n_groups=4, top_groups=0), H(top_k=4, group_top=3),
                H(top_k=5, n_groups=4, top_groups=1)):
        assert route(lib, bad) == nss.ERR_BAD_SHAPE
    assert route(lib, h, experts=1025) == nss.ERR_BAD_SHAPE
    assert route(lib, h, experts=0) == nss.ERR_BAD_SHAPE
    assert route(lib, h, tokens=-1) == nss.ERR_BAD_SHAPE
    assert route(lib, h, tokens=1 << 29) == nss.ERR_BAD_SHAPE
    assert route(lib, h, ld=15) == nss.ERR_BAD_SHAPE
    assert route(lib, h, ids=at(0) + 64) == nss.ERR_OVERLAP
    assert route(lib, h, w=at(1) + 32) == nss.ERR_OVERLAP
    assert route(lib, h, bias=at(1), w=at(2)) == nss.ERR_OVERLAP
    assert route(lib, h, tokens=0, logits=None, ids=None, w=None) == nss.OK
    with pytest.raises(TypeError):
        H(no_such_key=1)

    def back(h, d=at(3), dw=at(4), ld_d=16, ids=at(1)):
        return lib.muon_route_backward(dw, at(0), 0, 10, 16, 16, ids, ref(h), d, ld_d, None)
    assert back(None) == nss.ERR_NULL
    assert back(h, d=None) == nss.ERR_NULL
    assert back(h, dw=None) == nss.ERR_NULL
    assert back(h, ids=None) == nss.ERR_NULL
    assert back(h, ld_d=15) == nss.ERR_BAD_SHAPE
    assert back(h, d=at(3) + 1) == nss.ERR_ALIGN
    assert back(h, d=at(0)) == nss.ERR_OVERLAP


def test_order_refusals(lib):
    def run(n=100, E=8, align=16, cap=100 + 8 * 15, ids=at(0), off=at(1), cnt=at(2), rows=at(3), pos=at(4), ws=None, wsb=0):
        return lib.muon_expert_order(ids, n, E, align, off, cnt, rows, cap, pos, ws, wsb, None)
    for name in ("ids", "off", "cnt", "rows", "pos"):
        assert run(**{name: None}) == nss.ERR_NULL
        assert run(**{name: at(7) + 2}) == nss.ERR_ALIGN
    assert run(E=0) == nss.ERR_BAD_SHAPE
    assert run(E=1025, cap=1 << 20) == nss.ERR_BAD_SHAPE
    assert run(n=-1) == nss.ERR_BAD_SHAPE
    assert run(align=0) == nss.ERR_BAD_SHAPE
    assert run(align=1025, cap=1 << 20) == nss.ERR_BAD_SHAPE
    assert run(cap=100 + 8 * 15 - 1) == nss.ERR_RANGE
    assert run(cap=1 << 31) == nss.ERR_RANGE
    assert run(pos=at(0)) == nss.ERR_OVERLAP
    assert run(cnt=at(1) + 32) == nss.ERR_OVERLAP
    n = 1 << 17
    need = ctypes.c_size_t(0)
    assert lib.muon_expert_order_workspace_size(n, 8, ctypes.byref(need)) == nss.OK and need.value > 0
    assert run(n=n, cap=n + 200) == nss.ERR_NULL
    assert run(n=n, cap=n + 200, ws=at(5), wsb=need.value - 1) == nss.ERR_WORKSPACE
    assert run(n=n, cap=n + 200, ws=at(5) + 2, wsb=need.value) == nss.ERR_ALIGN
    assert run(n=n, cap=n + 200, ws=at(3), wsb=need.value) == nss.ERR_OVERLAP
    assert lib.muon_expert_order_workspace_size(n, 0, ctypes.byref(need)) == nss.ERR_BAD_SHAPE
    assert lib.muon_expert_order_workspace_size(n, 8, None) == nss.ERR_NULL


def test_combine_refusals(lib):
    def fwd(o=at(0), dtype=1, o_rows=60, cols=64, ld_o=64, pos=at(1), w=at(2), tokens=10, k=6, y=at(3), ld_y=64):
        return lib.muon_combine(o, dtype, o_rows, cols, ld_o, pos, w, tokens, k, y, ld_y, None)
    for name in ("o", "pos", "w", "y"):
        assert fwd(**{name: None}) == nss.ERR_NULL
        assert fwd(**{name: at(7) + 1}) == nss.ERR_ALIGN
    assert fwd(dtype=4) == nss.ERR_UNSUPPORTED
    for bad in (dict(k=0), dict(k=33), dict(tokens=-1), dict(tokens=1 << 29), dict(cols=-1), dict(o_rows=-1),
                dict(ld_o=63), dict(ld_y=63)):
        assert fwd(**bad) == nss.ERR_BAD_SHAPE
    assert fwd(y=at(0)) == nss.ERR_OVERLAP
    assert fwd(tokens=0, pos=None, w=None, y=None) == nss.OK

    def bwd(dy=at(0), o=at(1), pos=at(2), w=at(3), dw=at(4), do=at(5), tokens=10, ld_do=64):
        return lib.muon_combine_backward(dy, 1, tokens, 64, 64, o, 60, 64, pos, w, 6, dw, do, ld_do, None)
    for name in ("dy", "o", "pos", "w"):
        assert bwd(**{name: None}) == nss.ERR_NULL
    assert bwd(dw=None, do=None) == nss.ERR_NULL
    assert bwd(do=at(1)) == nss.ERR_OVERLAP
    assert bwd(dw=at(3)) == nss.ERR_OVERLAP
    assert bwd(ld_do=10) == nss.ERR_BAD_SHAPE
    assert bwd(tokens=0) == nss.OK


def test_operand_layout():
    import torch
    for rows, cols, pitch, sp in ((3, 1, 128, 4), (3, 128, 128, 4), (5, 129, 256, 4), (2, 513, 640, 8), (4, 0, 0, 0)):
        op = nss.fp8_empty(rows, cols, "e5m2", device="cpu")
        assert op.data.shape == (rows, pitch) and op.scale.shape == (rows, sp)
        assert op.rows == rows and op.cols == cols and op.format == "e5m2"
    op = nss.fp8_empty(3, 200, device="cpu", batch=2)
    assert op.data.shape == (2, 3, 256) and op.format == "e4m3"
    with pytest.raises(ValueError):
        nss.fp8_empty(3, 200, "e3m4", device="cpu")
    with pytest.raises(ValueError):
        nss.Fp8(op.data, op.scale, 300)
    with pytest.raises(ValueError):
        nss.Fp8(op.data, op.scale[:, :2], 200)
    with pytest.raises(TypeError):
        nss.Fp8(op.data.view(torch.uint8), op.scale, 200)
    with pytest.raises(ValueError):          # host tensors are refused
        nss.fp8_quantize(torch.zeros(4, 4))
    with pytest.raises(ValueError):
        nss.fp8_matmul(op, op)


def test_oracle_formats():
    import torch
    for fmt, td in (("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)):
        mine = F.decode_table(fmt)
        theirs = torch.arange(256, dtype=torch.uint8).view(td).double().numpy()
        assert np.array_equal(mine, theirs, equal_nan=True)
        rng = np.random.default_rng(0)
        top = 448.0 if fmt == "e4m3" else 57344.0
        x = np.concatenate([rng.uniform(-top, top, 2000), rng.standard_normal(2000) * 2.0 ** rng.integers(-20, 5, 2000),
                            mine[np.isfinite(mine)]]).astype(np.float32)
        x = x[np.abs(x) <= top]
        assert np.array_equal(F.round_to(x.astype(np.float64), fmt), torch.from_numpy(x).to(td).double().numpy())
        # the scale is the least that fits
        amax = np.abs(x[x != 0]).astype(np.float64)
        e = F.block_exponent(amax, fmt).astype(np.float64)
        assert np.all(amax <= top * 2.0 ** e) and np.all(amax > top * 2.0 ** (e - 1))


def test_oracle_order_and_route():
    off, cnt, rows, pos = R.expert_order(np.array([[2, 0], [2, -1], [0, 2]]), 3, 4, 20)
    assert off.tolist() == [0, 4, 4, 8] and cnt.tolist() == [2, 0, 3]
    assert rows[:8].tolist() == [1, 4, -1, -1, 0, 2, 5, -1] and pos.tolist() == [[4, 0], [5, -1], [1, 6]]
    ids, w = R.route(np.array([[0.0, 1.0, 1.0, -np.inf]]), 3)
    assert ids.tolist() == [[1, 2, 0]] and abs(w.sum() - 1) < 1e-15
