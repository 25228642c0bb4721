"""GPU: attention of so many tiles that queries of few sequences go one sequence after the other,
and that dK and dV take four waves per workgroup, in loops over many tiles.

Some heads are compared with the float64 oracle under the bounds of test_gpu_attention; all
heads with the same call behind empty sequences, whose tiles are listed beforehand; rows that
no sequence has keep what was in them.
"""
import numpy as np
import pytest

from test_gpu_attention import check_backward, check_forward, make

pytestmark = pytest.mark.gpu

LENS = [700, 0, 1, 333, 128, 129, 640, 257, 64, 511, 900, 350]
TILE, MANY = 128, 1024   # rows of a tile; tiles times heads from which on the order and the kernel are others
MARK = 9.0


def run(lib, off, q, k, v, do, **how):
    """(out, lse, dq, dk, dv), all of them filled with MARK before the calls."""
    import torch
    at = None if off is None else torch.from_numpy(np.asarray(off, np.int32)).cuda()
    out, dq, dk, dv = (torch.full_like(t, MARK) for t in (q, q, k, v))
    lse = torch.full((q.shape[1], q.shape[0]), MARK, device="cuda")
    lib.attention(q, k, v, offsets=at, out=out, lse=lse, **how)
    lib.attention_backward(do, q, k, v, out, lse, offsets=at, dq=dq, dk=dk, dv=dv, **how)
    return out, lse, dq, dk, dv


def compare(got, q, k, v, do, at, kv_heads, dtype, **how):
    out, lse, dq, dk, dv = got
    group = q.shape[1] // k.shape[1]
    for h in kv_heads:
        of, kv = slice(h * group, (h + 1) * group), slice(h, h + 1)
        part = [t[at, s] for t, s in ((q, of), (k, kv), (v, kv))]
        check_forward(*part, out[at, of], lse[of, at], dtype, **how)
        check_backward(do[at, of], *part, out[at, of], [dq[at, of], dk[at, kv], dv[at, kv]], dtype, **how)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads,kv,dim", [(32, 32, 32), (64, 32, 64), (27, 27, 96), (32, 32, 128)])
@pytest.mark.parametrize("window", [0, 150])
def test_many_tiles_of_few_sequences(lib, heads, kv, dim, window, dtype):
    import torch
    total = sum(LENS)
    T, off = total + 7, np.concatenate([[3], 3 + np.cumsum(LENS)])
    assert (T // TILE + len(LENS)) * kv >= MANY
    q, k, v, do = make(heads + dim, T, heads, kv, dim, dtype, loud=2.0)
    got = run(lib, off, q, k, v, do, causal=True, window=window)
    for t in got[:1] + got[2:]:
        assert (t[:3] == MARK).all() and (t[3 + total:] == MARK).all() and torch.isfinite(t).all()
    assert (got[1][:, :3] == MARK).all() and (got[1][:, 3 + total:] == MARK).all()
    at = slice(3, 3 + total)
    compare(got, q, k, v, do, at, (0, kv // 2, kv - 1), dtype, offsets=off - 3, causal=True, window=window)
    listed = run(lib, np.concatenate([off, np.full(70, off[-1])]), q, k, v, do, causal=True, window=window)
    assert all(torch.equal(a, b) for a, b in zip(got, listed))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,how", [(32, dict(causal=True)), (128, dict(causal=True)), (64, dict(causal=True, window=333)),
                                     (64, dict(causal=False))])
def test_many_tiles_of_one_sequence(lib, dim, how, dtype):
    import torch
    T, heads, kv = 2100, 128, 64
    assert -(-T // TILE) * kv >= MANY
    q, k, v, do = make(dim, T, heads, kv, dim, dtype, loud=2.0)
    got = run(lib, None, q, k, v, do, **how)
    compare(got, q, k, v, do, slice(0, T), (0, 41, 63), dtype, **how)
    packed = run(lib, [0, T], q, k, v, do, **how)   # the tile is found from the offsets
    assert all(torch.equal(a, b) for a, b in zip(got, packed))
