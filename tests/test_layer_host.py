"""The norm, embedding and clipping entry points without a GPU: every refusal, before any
device work (the addresses are never dereferenced)."""
import ctypes

import numpy as np
import pytest

import newton_schulz_step_amd as nss
from newton_schulz_step_amd import _binding as B
from oracle import layer as L

FAKE = 0x7f0000000000
GIB = 1 << 30
FAR = 64 * GIB


def at(i):
    return FAKE + i * FAR


@pytest.fixture(scope="module")
def lib():
    return nss.load()


def ref(x):
    return None if x is None else ctypes.byref(x)


def rows(**kw):
    f = dict(x=at(0), ld_x=300, residual=None, ld_residual=300, weight=at(2), rows=40, cols=300, dtype=1, weight_dtype=0,
             eps=1e-6, reserved=0)
    f.update(kw)
    return B.NormRows(*[f[n] for n, _ in B.NormRows._fields_])


def operand(i, r=40, c=300, batch=1, fmt=0, **kw):
    f = dict(data=at(i), scale=at(i) + 32 * GIB)
    f.update(kw)
    return B.Fp8Operand(f["data"], f["scale"], batch, r, c, fmt, 0)


def norm(lib, n, sum=None, ld_sum=300, y=at(4), ld_y=300, q=None, rstd=None):
    return lib.muon_rms_norm(ref(n), sum, ld_sum, y, ld_y, ref(q), rstd, None)


def test_norm_refusals(lib):
    assert norm(lib, None) == nss.ERR_NULL
    assert norm(lib, rows(x=None)) == nss.ERR_NULL
    assert norm(lib, rows(), y=None) == nss.ERR_NULL
    for bad in (dict(rows=-1), dict(rows=1 << 31), dict(cols=0), dict(cols=16385), dict(ld_x=-1), dict(ld_x=(1 << 28) + 1)):
        assert norm(lib, rows(**bad)) == nss.ERR_BAD_SHAPE, bad
    assert norm(lib, rows(), ld_y=299) == nss.ERR_BAD_SHAPE
    assert norm(lib, rows(residual=at(1)), sum=at(5), ld_sum=299) == nss.ERR_BAD_SHAPE
    for bad in (dict(dtype=3), dict(weight_dtype=-1), dict(dtype=-1)):
        assert norm(lib, rows(**bad)) == nss.ERR_UNSUPPORTED, bad
    for bad in (dict(x=at(0) + 1), dict(residual=at(1) + 1), dict(weight=at(2) + 2)):
        assert norm(lib, rows(**bad)) == nss.ERR_ALIGN, bad
    assert norm(lib, rows(), y=at(4) + 1) == nss.ERR_ALIGN
    assert norm(lib, rows(), rstd=at(6) + 2) == nss.ERR_ALIGN
    for eps in (-1e-9, float("nan"), float("inf")):
        assert norm(lib, rows(eps=eps)) == nss.ERR_BAD_HYPER
    assert norm(lib, rows(), y=at(0) + 600) == nss.ERR_OVERLAP
    assert norm(lib, rows(), y=at(2)) == nss.ERR_OVERLAP
    assert norm(lib, rows(residual=at(1)), sum=at(1)) == nss.ERR_OVERLAP
    assert norm(lib, rows(), sum=at(4)) == nss.ERR_OVERLAP
    for q in (operand(6, 41), operand(6, 40, 301), operand(6, batch=2)):
        assert norm(lib, rows(), q=q) == nss.ERR_BAD_SHAPE
    assert norm(lib, rows(), q=operand(6, fmt=2)) == nss.ERR_UNSUPPORTED
    assert norm(lib, rows(), q=operand(6, data=at(6) + 8)) == nss.ERR_ALIGN
    assert norm(lib, rows(), q=operand(6, data=None)) == nss.ERR_NULL
    assert norm(lib, rows(rows=0)) == nss.OK


def back(lib, n, rstd=at(3), dy=at(5), ld_dy=300, dsum=None, ld_dsum=300, dx=at(6), ld_dx=300, dw=at(7), dw_type=0,
         acc=0, ws=at(8), ws_bytes=1 << 30):
    return lib.muon_rms_norm_backward(ref(n), rstd, dy, ld_dy, dsum, ld_dsum, dx, ld_dx, dw, dw_type, acc, ws, ws_bytes, None)


def test_norm_gradient_refusals(lib):
    assert back(lib, None) == nss.ERR_NULL
    assert back(lib, rows(), dx=None, dw=None) == nss.ERR_NULL
    assert back(lib, rows(), rstd=None) == nss.ERR_NULL
    assert back(lib, rows(), dy=None) == nss.ERR_NULL
    assert back(lib, rows(), ws=None) == nss.ERR_NULL
    assert back(lib, rows(residual=at(1))) == nss.ERR_UNSUPPORTED
    assert back(lib, rows(), dw_type=5) == nss.ERR_UNSUPPORTED
    need = nss.rms_norm_backward_workspace_size(40, 300)
    assert need >= 300 * 4
    assert back(lib, rows(), ws_bytes=need - 1) == nss.ERR_WORKSPACE
    assert back(lib, rows(), ws=at(8) + 2) == nss.ERR_ALIGN
    assert back(lib, rows(), rstd=at(3) + 2) == nss.ERR_ALIGN
    assert back(lib, rows(), ld_dx=10) == nss.ERR_BAD_SHAPE
    assert back(lib, rows(), dx=at(5)) == nss.ERR_OVERLAP
    assert back(lib, rows(), ws=at(0)) == nss.ERR_OVERLAP
    assert back(lib, rows(), dsum=at(6)) == nss.ERR_OVERLAP
    with pytest.raises(nss.MuonError):
        nss.rms_norm_backward_workspace_size(-1, 8)
    with pytest.raises(nss.MuonError):
        nss.rms_norm_backward_workspace_size(1, 16385)


def tokens(**kw):
    f = dict(ids=at(0), tokens=100, vocab=50, cols=64, ld=64, id_bytes=8, table_dtype=0, scale=1.0, reserved=0)
    f.update(kw)
    return B.EmbeddingTokens(*[f[n] for n, _ in B.EmbeddingTokens._fields_])


def look(lib, e, table=at(1), y=at(2), dtype=1, ld_y=64):
    return lib.muon_embedding(ref(e), table, y, dtype, ld_y, None)


def look_back(lib, e, dy=at(1), dtype=1, ld_dy=64, dtable=at(2), acc=0, ws=at(3), ws_bytes=1 << 30):
    return lib.muon_embedding_backward(ref(e), dy, dtype, ld_dy, dtable, acc, ws, ws_bytes, None)


def test_embedding_refusals(lib):
    for call in (look, look_back):
        assert call(lib, None) == nss.ERR_NULL
        assert call(lib, tokens(ids=None)) == nss.ERR_NULL
        for bad in (dict(tokens=-1), dict(tokens=1 << 31), dict(vocab=0), dict(vocab=(1 << 30) + 1), dict(cols=-1),
                    dict(cols=1 << 23), dict(ld=(1 << 28) + 1)):
            assert call(lib, tokens(**bad)) == nss.ERR_BAD_SHAPE, bad
        for bad in (dict(id_bytes=2), dict(id_bytes=0), dict(table_dtype=3)):
            assert call(lib, tokens(**bad)) == nss.ERR_UNSUPPORTED, bad
        assert call(lib, tokens(), dtype=7) == nss.ERR_UNSUPPORTED
        assert call(lib, tokens(ids=at(0) + 4)) == nss.ERR_ALIGN
        for scale in (float("nan"), float("inf")):
            assert call(lib, tokens(scale=scale)) == nss.ERR_BAD_HYPER
    assert look(lib, tokens(), table=None) == nss.ERR_NULL
    assert look(lib, tokens(), y=None) == nss.ERR_NULL
    assert look(lib, tokens(), ld_y=63) == nss.ERR_BAD_SHAPE
    assert look(lib, tokens(), y=at(1)) == nss.ERR_OVERLAP
    assert look(lib, tokens(), y=at(0)) == nss.ERR_OVERLAP
    assert look(lib, tokens(tokens=0, ids=None)) == nss.OK
    assert look_back(lib, tokens(), dy=None) == nss.ERR_NULL
    assert look_back(lib, tokens(), dtable=None) == nss.ERR_NULL
    assert look_back(lib, tokens(), ws=None) == nss.ERR_NULL
    assert look_back(lib, tokens(ld=63)) == nss.ERR_BAD_SHAPE
    need = nss.embedding_backward_workspace_size(100, 50, 64)
    assert look_back(lib, tokens(), ws_bytes=need - 1) == nss.ERR_WORKSPACE
    assert look_back(lib, tokens(), ws=at(3) + 8) == nss.ERR_ALIGN
    assert look_back(lib, tokens(), dtable=at(1)) == nss.ERR_OVERLAP
    assert look_back(lib, tokens(), ws=at(2)) == nss.ERR_OVERLAP
    assert look_back(lib, tokens(), ws=at(0)) == nss.ERR_OVERLAP
    with pytest.raises(nss.MuonError):
        nss.embedding_backward_workspace_size(-1, 50, 64)


def tensors(*ts):
    flat = [v for t in ts for v in t]
    return (ctypes.c_int64 * max(1, len(flat)))(*flat), len(ts)


def clip(lib, ins, outs=None, sumsq=at(8), max_norm=1.0, norm=at(9)):
    a, n = tensors(*ins)
    return lib.muon_grad_clip(a, None if outs is None else tensors(*outs)[0], n, sumsq, max_norm, norm, None)


def sumsq(lib, ins, out=at(8), ws=at(9), ws_bytes=1 << 30, n=None):
    a, m = tensors(*ins)
    return lib.muon_grad_sumsq(a, m if n is None else n, 0, out, ws, ws_bytes, None)


def test_clip_refusals(lib):
    ok = (at(0), 1000, 0)
    for call in (clip, sumsq):
        assert call(lib, [ok, (0, 10, 0)]) == nss.ERR_NULL
        assert call(lib, [ok, (at(1), 10, 3)]) == nss.ERR_UNSUPPORTED
        assert call(lib, [(at(1) + 2, 10, 0)]) == nss.ERR_ALIGN
        assert call(lib, [(at(1), -1, 0)]) == nss.ERR_BAD_SHAPE
        assert call(lib, [(at(1), (1 << 36) + 1, 0)]) == nss.ERR_BAD_SHAPE
        assert call(lib, [(at(1), 1 << 36, 1), (at(4), 1, 1)]) == nss.ERR_BAD_SHAPE
    assert sumsq(lib, [ok], n=-1) == nss.ERR_BAD_SHAPE
    assert sumsq(lib, [ok], n=(1 << 20) + 1) == nss.ERR_BAD_SHAPE
    assert lib.muon_grad_sumsq(None, 1, 0, at(8), at(9), 1 << 30, None) == nss.ERR_NULL
    assert sumsq(lib, [ok], out=None) == nss.ERR_NULL
    assert sumsq(lib, [ok], ws=None) == nss.ERR_NULL
    assert sumsq(lib, [ok], out=at(8) + 4) == nss.ERR_ALIGN
    assert sumsq(lib, [ok], ws=at(9) + 4) == nss.ERR_ALIGN
    assert sumsq(lib, [ok], ws_bytes=7) == nss.ERR_WORKSPACE
    assert sumsq(lib, [ok], out=at(0) + 8) == nss.ERR_OVERLAP
    assert sumsq(lib, [ok], ws=at(0)) == nss.ERR_OVERLAP
    assert clip(lib, [ok], sumsq=None) == nss.ERR_NULL
    assert clip(lib, [ok], sumsq=at(8) + 4) == nss.ERR_ALIGN
    assert clip(lib, [ok], norm=at(9) + 2) == nss.ERR_ALIGN
    for bad in (-1.0, float("nan")):
        assert clip(lib, [ok], max_norm=bad) == nss.ERR_BAD_HYPER
    assert clip(lib, [ok], [(at(1), 999, 0)]) == nss.ERR_BAD_SHAPE
    two = [ok, (at(1), 1000, 0)]
    assert clip(lib, two, [(at(2), 1000, 1), (at(2) + 1998, 1000, 1)]) == nss.ERR_OVERLAP    # outputs
    assert clip(lib, two, [(at(1), 1000, 0), (at(2), 1000, 0)]) == nss.ERR_OVERLAP           # another one's input
    assert clip(lib, two, [(at(0), 1000, 1), (at(2), 1000, 0)]) == nss.ERR_OVERLAP           # its own, of another type
    assert clip(lib, two, [(at(0) + 4, 1000, 0), (at(2), 1000, 0)]) == nss.ERR_OVERLAP
    assert clip(lib, [ok, ok]) == nss.ERR_OVERLAP                                            # one tensor twice, in place
    assert clip(lib, [ok], norm=at(0) + 8) == nss.ERR_OVERLAP
    assert clip(lib, [ok], sumsq=at(0) + 8) == nss.ERR_OVERLAP


def test_binding_refusals():
    import torch
    x, w = torch.zeros(4, 8), torch.ones(8)
    with pytest.raises(ValueError, match="on a GPU"):
        nss.rms_norm(x, w)
    with pytest.raises(ValueError, match="fp8"):
        nss.rms_norm(x, w, fp8="yes")
    with pytest.raises(ValueError, match="format"):
        nss.rms_norm(x, w, fmt="e3m4")
    with pytest.raises(ValueError, match="weight"):
        nss.rms_norm(x, torch.ones(7))
    with pytest.raises(ValueError, match="residual"):
        nss.rms_norm(x, w, residual=torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="does not make"):
        nss.rms_norm(x, w, out_sum=x)
    with pytest.raises(ValueError, match="last dimension"):
        nss.rms_norm(torch.zeros(8, 4).t(), w)
    with pytest.raises(TypeError, match="dtype"):
        nss.rms_norm(x.double(), w)
    with pytest.raises(ValueError, match="rows, cols"):
        nss.embedding(torch.zeros(3, dtype=torch.int32), torch.zeros(3))
    with pytest.raises(ValueError, match="shape of ids"):
        nss.embedding_backward(torch.zeros(3, 8), torch.zeros(4, dtype=torch.int32), 9)
    with pytest.raises(ValueError, match="share one GPU"):
        nss.clip_gradients([x], 1.0)
    with pytest.raises(ValueError, match="at least one"):
        nss.clip_gradients([], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        nss.grad_sumsq([torch.zeros(4, 8).t()])
    with pytest.raises(ValueError, match="rstd"):
        nss.rms_norm_backward(x, x, w, torch.ones(3))
    with pytest.raises(ValueError, match="without a weight"):
        nss.rms_norm_backward(x, x, None, torch.ones(4), dweight=w)


def test_oracle_against_differences():
    rng = np.random.default_rng(0)
    x, w, dy = rng.standard_normal((3, 10)), rng.standard_normal(10), rng.standard_normal((3, 10))
    dx, dw = L.rms_norm_backward(dy, x, w, L.rms_norm(x, w)[1])
    h = 1e-6
    for a, g in ((x, dx), (w, dw)):
        for i in np.ndindex(*a.shape):
            keep = a[i]
            a[i] = keep + h
            up = np.sum(dy * L.rms_norm(x, w)[0])
            a[i] = keep - h
            down = np.sum(dy * L.rms_norm(x, w)[0])
            a[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) < 1e-6
