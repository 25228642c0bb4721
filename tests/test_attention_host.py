"""The attention entry points without a GPU: every refusal, before any device work (the
addresses are never dereferenced), and the oracle's gradient against differences."""
import ctypes

import numpy as np
import pytest

import newton_schulz_step_amd as nss
from newton_schulz_step_amd import _binding as B
from oracle import layer as L

FAKE = 0x7f0000000000
FAR = 64 << 30


def at(i):
    return FAKE + i * FAR


@pytest.fixture(scope="module")
def lib():
    return nss.load()


def rows(**kw):
    f = dict(tokens=100, offsets=None, sequences=0, heads=8, kv_heads=2, dim=64, dtype=1, causal=1, window=0, scale=0.125)
    f.update(kw)
    return B.AttentionRows(*[f[n] for n, _ in B.AttentionRows._fields_])


def heads(i, ts=512, hs=64, data=None):
    return B.Heads(at(i) if data is None else data, ts, hs)


def ref(x):
    return None if x is None else ctypes.byref(x)


def forward(lib, a=None, q=heads(0), k=heads(1), v=heads(2), o=heads(3), lse=at(4), ws=at(5), ws_bytes=1 << 30):
    return lib.muon_attention(ref(rows() if a is None else a), ref(q), ref(k), ref(v), ref(o), lse, ws, ws_bytes, None)


def backward(lib, a=None, d_o=heads(10), q=heads(0), k=heads(1), v=heads(2), o=heads(3), lse=at(4), dq=heads(6),
             dk=heads(7), dv=heads(8), ws=at(5), ws_bytes=1 << 30):
    return lib.muon_attention_backward(ref(rows() if a is None else a), ref(d_o), ref(q), ref(k), ref(v), ref(o), lse,
                                       ref(dq), ref(dk), ref(dv), ws, ws_bytes, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_refusals_of_both(lib, call):
    for bad in (dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(heads=0), dict(heads=1025, kv_heads=1), dict(kv_heads=0),
                dict(kv_heads=3), dict(kv_heads=16), dict(dim=0), dict(dim=4), dict(dim=60), dict(dim=136), dict(window=-1),
                dict(offsets=at(9), sequences=-1)):
        assert call(lib, rows(**bad)) == nss.ERR_BAD_SHAPE, bad
    for bad in (dict(dtype=0), dict(dtype=3), dict(causal=0, window=5)):
        assert call(lib, rows(**bad)) == nss.ERR_UNSUPPORTED, bad
    for scale in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert call(lib, rows(scale=scale)) == nss.ERR_BAD_HYPER
    assert call(lib, rows(offsets=at(9) + 2, sequences=3)) == nss.ERR_ALIGN
    for n in ("q", "k", "v", "o"):
        assert call(lib, **{n: heads(0, data=0)}) == nss.ERR_NULL
        assert call(lib, **{n: heads(0, data=at(0) + 8)}) == nss.ERR_ALIGN
        assert call(lib, **{n: heads(0, ts=516)}) == nss.ERR_ALIGN
        assert call(lib, **{n: heads(0, hs=68)}) == nss.ERR_ALIGN
        assert call(lib, **{n: heads(0, ts=56)}) == nss.ERR_BAD_SHAPE
        assert call(lib, **{n: heads(0, ts=(1 << 22) + 8)}) == nss.ERR_BAD_SHAPE
        assert call(lib, **{n: heads(0, hs=-64)}) == nss.ERR_BAD_SHAPE
    assert call(lib, lse=at(4) + 2) == nss.ERR_ALIGN
    assert call(lib, rows(offsets=at(9), sequences=65), ws=None) == nss.ERR_NULL
    assert call(lib, rows(offsets=at(9), sequences=65), ws_bytes=15) == nss.ERR_WORKSPACE
    assert call(lib, rows(offsets=at(9), sequences=65), ws=at(5) + 8) == nss.ERR_ALIGN
    assert call(lib, rows(tokens=0)) == nss.OK


def test_null_descriptions(lib):
    assert lib.muon_attention(None, None, None, None, None, None, None, 0, None) == nss.ERR_NULL
    assert forward(lib, q=None) == nss.ERR_NULL
    assert backward(lib, dv=None) == nss.ERR_NULL
    assert backward(lib, lse=None) == nss.ERR_NULL
    n = ctypes.c_size_t(0)
    assert lib.muon_attention_workspace_size(ctypes.byref(rows()), 0, None) == nss.ERR_NULL
    assert lib.muon_attention_workspace_size(None, 0, ctypes.byref(n)) == nss.ERR_NULL
    assert lib.muon_attention_workspace_size(ctypes.byref(rows()), 0, ctypes.byref(n)) == nss.OK and n.value == 0
    assert lib.muon_attention_workspace_size(ctypes.byref(rows()), 1, ctypes.byref(n)) == nss.OK and n.value >= 2 * 800 * 4


def test_overlaps(lib):
    assert forward(lib, o=heads(0)) == nss.ERR_OVERLAP
    assert forward(lib, o=heads(0, data=at(2) + 64)) == nss.ERR_OVERLAP
    assert forward(lib, lse=at(3) + 128) == nss.ERR_OVERLAP
    assert forward(lib, rows(offsets=at(9), sequences=65), ws=at(0)) == nss.ERR_OVERLAP
    assert forward(lib, rows(offsets=at(9), sequences=65), ws=at(9)) == nss.ERR_OVERLAP
    assert forward(lib, rows(offsets=at(3), sequences=3)) == nss.ERR_OVERLAP
    assert forward(lib, o=heads(3, ts=64, hs=64)) == nss.ERR_BAD_SHAPE          # heads on top of tokens
    assert forward(lib, o=heads(3, ts=512, hs=32)) == nss.ERR_BAD_SHAPE
    assert backward(lib, dq=heads(7)) == nss.ERR_OVERLAP
    assert backward(lib, dk=heads(10)) == nss.ERR_OVERLAP
    assert backward(lib, ws=at(8)) == nss.ERR_OVERLAP
    # parts of one gradient: columns [0, 512), [512, 640), [640, 768) of rows of 768; one column block off they meet
    part = [dict(ts=768, data=at(6) + 2 * c) for c in (0, 512, 640, 632)]
    assert backward(lib, dq=heads(6, **part[0]), dk=heads(6, **part[0]), dv=heads(6, **part[2])) == nss.ERR_OVERLAP
    assert backward(lib, dq=heads(6, **part[0]), dk=heads(6, **part[1]), dv=heads(6, **part[3])) == nss.ERR_OVERLAP
    other = heads(6, ts=776, data=at(6) + 2 * 512)                                # another pitch
    assert backward(lib, dq=heads(6, **part[0]), dk=other) == nss.ERR_OVERLAP


def test_overlaps_of_parts_of_heads(lib):
    """dq, dk, dv of every head next to each other; a column too near, a pitch that is no multiple of the heads', heads
    at other distances: refused."""
    def call(dk=64, dv=128, ts=8 * 192, hs=(192, 192, 192), tokens=100):
        part = [B.Heads(at(6) + 2 * c, ts, h) for c, h in zip((0, dk, dv), hs)]
        return backward(lib, rows(kv_heads=8, tokens=tokens), dq=part[0], dk=part[1], dv=part[2], ws=at(6))
    # where they are apart, the workspace, which begins at dq, is what is refused
    for good in (dict(), dict(tokens=1), dict(tokens=1, ts=64)):
        assert call(**good) == nss.ERR_OVERLAP and b"workspace" in lib.muon_last_error(), good
    for bad in (dict(dk=56), dict(dv=136), dict(dv=64), dict(ts=8 * 192 + 8), dict(hs=(192, 192, 200), ts=8 * 200),
                dict(tokens=1, dk=56)):
        assert call(**bad) == nss.ERR_OVERLAP and b"workspace" not in lib.muon_last_error(), bad


def test_binding_refusals():
    import torch
    q, k = torch.zeros(6, 4, 64, dtype=torch.bfloat16), torch.zeros(6, 2, 64, dtype=torch.bfloat16)
    lse = torch.zeros(4, 6)
    with pytest.raises(ValueError, match="on a GPU"):
        nss.attention(q, k, k)
    with pytest.raises(ValueError, match="kv_heads"):
        nss.attention(q, k, k[:5])
    with pytest.raises(TypeError, match="one type"):
        nss.attention(q, k, k.half())
    with pytest.raises(ValueError, match="int32"):
        nss.attention(q, k, k, offsets=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="one element more"):
        nss.attention(q, k, k, offsets=torch.zeros(0, dtype=torch.int32))
    with pytest.raises(ValueError, match="out must be"):
        nss.attention_backward(q, q, k, k, q[:, :2], lse)
    with pytest.raises(ValueError, match="lse"):
        nss.attention_backward(q, q, k, k, q, lse[:2])


def test_oracle_against_differences():
    r = np.random.default_rng(0)
    q, k, v, do = (r.standard_normal((9, h, 8)) for h in (4, 2, 2, 4))
    how = dict(offsets=[0, 4, 9], window=3)
    for a, g in zip((q, k, v), L.attention_backward(do, q, k, v, **how)):
        for i in [(0, 0, 0), (3, 1, 5), (8, 0, 7), (6, 1, 2)]:
            keep, h = a[i], 1e-6
            a[i] = keep + h
            up = np.sum(do * L.attention(q, k, v, **how)[0])
            a[i] = keep - h
            down = np.sum(do * L.attention(q, k, v, **how)[0])
            a[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) < 1e-7
