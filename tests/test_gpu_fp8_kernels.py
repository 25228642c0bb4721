"""GPU: every kernel of the products with the values, types and forms that it serves. The
launch statistics say which kernel ran, so that a change of the choice among them cannot take
a case away from it. Bounds as in test_gpu_fp8.py.

The few-row kernel has one name for its three heights; the sizes below take 16, 32 and 64 rows
by the cost table.
"""
import numpy as np
import pytest

from test_gpu_fp8 import check_product, dt, host, kinds, operand, values

pytestmark = pytest.mark.gpu

FORMATS = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")]
# rows, columns, contraction: cut and whole tiles of every kernel
SIZES = [(5, 40, 300, "few_rows"), (50, 5000, 700, "few_rows"), (64, 3000, 2100, "few_rows"),
         (1030, 1000, 1500, "128"), (1024, 1024, 1536, "128"), (2100, 4000, 260, "256"), (2304, 4096, 256, "256")]


def pick(rng, n, most=150):
    """Some rows: the first, the last, and a few in between."""
    return np.unique(np.concatenate([[0, n - 1], rng.integers(0, n, most)]))


def scaled(lib, rng, rows, cols, fmt, spread):
    """An operand whose scales differ from block to block by up to 2^(2 spread)."""
    import torch
    x = rng.standard_normal((rows, cols))
    for k in range(0, cols, 128):
        x[:, k:k + 128] *= 2.0 ** rng.integers(-spread, spread + 1, (rows, 1))
    op = lib.fp8_quantize(torch.from_numpy(x.astype(np.float32)).cuda(), fmt)
    return op, values(op)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fa,fb", FORMATS)
@pytest.mark.parametrize("M,N,K,kernel", SIZES)
def test_dense(lib, M, N, K, kernel, fa, fb, dtype):
    # per-block scales, results into a view with an odd offset and pitch, then added to it
    import torch
    rng = np.random.default_rng([M, N, len(dtype)])
    spread = 2 if dtype == "f16" else 20        # fp16 results stay in range
    a, va = scaled(lib, rng, M, K, fa, spread)
    b, vb = scaled(lib, rng, N, K, fb, spread)
    rows, cols = pick(rng, M), pick(rng, N)
    for off, pitch in ((3, N + 5), (0, N)):
        buf = torch.full((off + M * pitch,), 7.0, dtype=dt(torch, dtype), device="cuda")
        out = buf[off:].as_strided((M, N), (pitch, 1))
        assert kinds(lib, lambda: lib.fp8_matmul(a, b, out=out)) == {"fp8_gemm_" + kernel}
        first = host(out)
        check_product(first[np.ix_(rows, cols)], va[rows], vb[cols], dtype)
        assert kinds(lib, lambda: lib.fp8_matmul(a, b, out=out, accumulate=True)) == {"fp8_gemm_" + kernel}
        check_product(host(out)[np.ix_(rows, cols)], va[rows], vb[cols], dtype, first[np.ix_(rows, cols)])
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask.as_strided((M, N), (pitch, 1), off).fill_(False)
        assert torch.all(buf[mask] == 7.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K,kernel", SIZES)
def test_nan_and_inf_stay_in_their_rows(lib, M, N, K, kernel, dtype):
    import torch
    rng = np.random.default_rng(M)
    x, w = rng.standard_normal((M, K)).astype(np.float32), rng.standard_normal((N, K)).astype(np.float32)
    x[3, 7], x[1, 200], w[11, 5] = np.nan, np.inf, np.nan
    a, b = lib.fp8_quantize(torch.from_numpy(x).cuda(), "e5m2"), lib.fp8_quantize(torch.from_numpy(w).cuda())
    out = torch.empty(M, N, dtype=dt(torch, dtype), device="cuda")
    assert kinds(lib, lambda: lib.fp8_matmul(a, b, out=out)) == {"fp8_gemm_" + kernel}
    got = host(out)
    assert np.all(np.isnan(got[3])) and np.all(np.isnan(got[:, 11])) and not np.any(np.isfinite(got[1]))
    rows, cols = (np.setdiff1d(pick(rng, n), bad) for n, bad in ((M, [1, 3]), (N, [11])))
    check_product(got[np.ix_(rows, cols)], values(a)[rows], values(b)[cols], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,kernel", [(1500, 1500, "128"), (4096, 4000, "256")])
def test_more_blocks_than_the_parts_of_the_scales_hold(lib, M, N, kernel, dtype):
    # 81 blocks, 16 in a part, the last one of a single block
    import torch
    rng = np.random.default_rng(N)
    K = 128 * 80 + 5
    a, va = scaled(lib, rng, M, K, "e4m3", 3)
    b, vb = scaled(lib, rng, N, K, "e4m3", 3)
    out = torch.empty(M, N, dtype=dt(torch, dtype), device="cuda")
    assert kinds(lib, lambda: lib.fp8_matmul(a, b, out=out)) == {"fp8_gemm_" + kernel}
    rows, cols = pick(rng, M, 60), pick(rng, N, 60)
    check_product(host(out)[np.ix_(rows, cols)], va[rows], vb[cols], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N,groups,kernel", [(260, 300, 70, "128"), (1030, 1000, 8, "256")])
def test_last_tile_fetches_nothing_more(lib, M, N, groups, kernel, accumulate, dtype):
    # the last tiles' contraction begins in the middle of the operands (beyond the first 16
    # blocks too) and ends with their last block; behind it a workgroup fetches nothing
    import torch
    rng = np.random.default_rng([M, 26])
    off = ([0, 1, 19, 20] + [20] * groups)[:groups - 3] + [20, 21, 36, 37]
    assert len(off) == groups + 1
    a, va = operand(lib, rng, M, 128 * 37, "e4m3")
    b, vb = operand(lib, rng, N, 128 * 37, "e5m2")
    out = torch.full((groups, M, N), 0.5, dtype=dt(torch, dtype), device="cuda")
    offsets = (128 * torch.tensor(off, dtype=torch.int32)).cuda()
    call = lambda: lib.fp8_matmul_grouped_k(a, b, offsets, out=out, accumulate=accumulate)   # noqa: E731
    assert kinds(lib, call) == {"fp8_gemm_" + kernel}
    rows = pick(rng, M, 60)
    got = host(out[:, torch.from_numpy(rows).cuda()])
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        check_product(got[g], va[rows, 128 * lo:128 * hi], vb[:, 128 * lo:128 * hi], dtype,
                      np.full((1, 1), 0.5) if accumulate else None)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K,G,kernel", [(300, 60, 200, 5, "few_rows"), (1500, 1300, 520, 7, "128"),
                                            (9000, 3000, 136, 9, "256")])
def test_groups_of_rows(lib, M, N, K, G, kernel, dtype):
    # e5m2 on both sides, every type, stored and added; rows outside all groups stay
    import torch
    rng = np.random.default_rng([M, G])
    s = 2.0 ** -8 if dtype == "f16" else 1.0
    a = lib.fp8_quantize(torch.from_numpy((operand(lib, rng, M, K, "e5m2")[1] * s).astype(np.float32)).cuda(), "e5m2")
    va = values(a)
    b, vb = operand(lib, rng, N, K, "e5m2", G)
    off = np.sort(rng.integers(0, M, G + 1))
    off[2] = off[1]
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    out = torch.full((M, N), 7.0, dtype=dt(torch, dtype), device="cuda")
    cols = pick(rng, N, 40)
    for accumulate in (False, True):
        base = host(out)[:, cols]
        call = lambda: lib.fp8_matmul(a, b, out=out, offsets=offsets, accumulate=accumulate)   # noqa: E731, B023
        assert kinds(lib, call) == {"fp8_gemm_" + kernel}
        got = host(out)[:, cols]
        for g in range(G):
            at = slice(off[g], off[g + 1])
            check_product(got[at], va[at], vb[g][cols], dtype, base[at] if accumulate else None)
        assert np.all(got[:off[0]] == 7.0) and np.all(got[off[-1]:] == 7.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(3, 40), (1100, 1000), (8000, 8100)])
def test_no_terms(lib, M, N, dtype):
    # a contraction of length zero, on all kernels: zeros, or what is there
    import torch
    for a, b, shape, kw in ((lib.fp8_empty(M, 0), lib.fp8_empty(N, 0), (M, N), {}),
                            (lib.fp8_empty(M, 0), lib.fp8_empty(N, 0, batch=2), (M, N),
                             dict(offsets=torch.tensor([0, M // 2, M], dtype=torch.int32).cuda()))):
        out = torch.full(shape, 3.0, dtype=dt(torch, dtype), device="cuda")
        lib.fp8_matmul(a, b, out=out, accumulate=True, **kw)
        assert torch.all(out == 3.0)
        lib.fp8_matmul(a, b, out=out, **kw)
        assert torch.all(out == 0.0)
