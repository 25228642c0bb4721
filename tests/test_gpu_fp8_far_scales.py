"""GPU: fp32 results of operands whose scales lie at the ends of their range, where values
times scales do not fit into the 16-bit numbers that are multiplied. The products themselves
are ordinary numbers (no product is subnormal, no sum overflows), so the bound of
test_gpu_fp8.py holds: a block's own sum, its factor (a power of two: exact) and one more
addition per block of 128 make at most K + 16 additions for K up to 2048.
"""
import numpy as np
import pytest

from test_gpu_fp8 import check_product, host, kinds, operand, values

pytestmark = pytest.mark.gpu

FORMATS = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")]


def shift(op, by):
    """Adds `by` (rows x blocks) to the scales' exponents, kept in bytes 0 .. 254."""
    import torch
    s = op.scale.view(torch.uint8)
    blocks = op.data.shape[-1] // 128
    e = s[..., :blocks].cpu().numpy().astype(np.int64) + by
    s[..., :blocks] = torch.from_numpy(np.clip(e, 0, 254).astype(np.uint8)).cuda()


def far_pair(lib, rng, M, N, K, fa, fb, batch=None, both=False):
    """Operands of ordinary blocks and of blocks whose scales lie on both sides of the
    lower or of the upper border: in bands of A's rows, met by scales of B far the other way
    but in range, or (`both`) in all rows, met by ones at B's own border. The last of several
    blocks is ordinary."""
    a, _ = operand(lib, rng, M, K, fa)
    b, _ = operand(lib, rng, N, K, fb, batch)
    blocks = -(-K // 128)
    kind = rng.integers(-1, 2, blocks)
    kind[0] = rng.choice([-1, 1])
    if blocks > 1:
        kind[-1] = 0
    low, high = (-112, 122) if fa == "e4m3" else (-100, 126)
    by_a = np.where(kind < 0, low, np.where(kind > 0, high, 0)) + np.zeros((M, 1), np.int64)
    lead = () if batch is None else (batch,)
    by_b = (-by_a[:1] if both else -90 * kind) + np.zeros(lead + (N, 1), np.int64)
    if not both:
        by_a[np.arange(M) // 40 % 3 != 0] = 0
    shift(a, by_a)
    shift(b, by_b)
    return a, values(a), b, values(b)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("M,N,K,kernel", [(5, 40, 300, "few_rows"), (30, 200, 1000, "few_rows"), (60, 500, 640, "few_rows"),
                                          (1030, 1000, 1500, "128"), (1024, 1024, 1500, "128"), (2100, 4000, 260, "256")])
def test_dense(lib, M, N, K, kernel, accumulate):
    import torch
    for turn, (fa, fb) in enumerate(FORMATS if M < 1000 or not accumulate else FORMATS[:1]):
        rng = np.random.default_rng([M, turn])
        a, va, b, vb = far_pair(lib, rng, M, N, K, fa, fb, both=turn % 2 == 1)
        out = torch.full((M, N), 0.5, device="cuda")
        assert kinds(lib, lambda: lib.fp8_matmul(a, b, out=out, accumulate=accumulate)) == {"fp8_gemm_" + kernel}
        rows, cols = np.arange(0, M, 1 + M // 200), np.arange(0, N, 1 + N // 200)
        got = host(out)[np.ix_(rows, cols)]
        check_product(got, va[rows], vb[cols], "f32", np.full((1, 1), 0.5) if accumulate else None)


@pytest.mark.parametrize("M,N,K,G,kernel", [(300, 40, 200, 4, "few_rows"), (1500, 1300, 520, 7, "128"),
                                            (4000, 3000, 136, 9, "256")])
def test_grouped_rows(lib, M, N, K, G, kernel):
    import torch
    rng = np.random.default_rng([M, G])
    a, va, b, vb = far_pair(lib, rng, M, N, K, "e4m3", "e5m2", G)
    off = np.sort(rng.integers(0, M, G + 1))
    out = torch.full((M, N), 7.0, device="cuda")
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    assert kinds(lib, lambda: lib.fp8_matmul(a, b, out=out, offsets=offsets)) == {"fp8_gemm_" + kernel}
    cols = rng.permutation(N)[:40]
    got = host(out)[:, cols]
    for g in range(G):
        check_product(got[off[g]:off[g + 1]], va[off[g]:off[g + 1]], vb[g][cols], "f32")
    assert np.all(got[:off[0]] == 7.0) and np.all(got[off[-1]:] == 7.0)


@pytest.mark.parametrize("M,N,blocks,G,kernel", [(20, 40, 9, 5, "few_rows"), (300, 260, 100, 70, "128"),
                                                 (1024, 1000, 30, 70, "256")])
def test_grouped_contraction(lib, M, N, blocks, G, kernel):
    import torch
    rng = np.random.default_rng([M, G])
    a, va, b, vb = far_pair(lib, rng, M, N, 128 * blocks, "e5m2", "e4m3")
    off = np.sort(rng.integers(0, blocks + 1, G + 1)) * 128
    out = torch.full((G, M, N), 7.0, device="cuda")
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    assert kinds(lib, lambda: lib.fp8_matmul_grouped_k(a, b, offsets, out=out)) == {"fp8_gemm_" + kernel}
    rows = np.arange(0, M, 1 + M // 20)
    got = host(out[:, torch.from_numpy(rows).cuda()])
    for g in range(G):
        check_product(got[g], va[rows, off[g]:off[g + 1]], vb[:, off[g]:off[g + 1]], "f32")


@pytest.mark.parametrize("M,N", [(4, 40), (1024, 1024)])
def test_quantised_ends_of_fp32(lib, M, N):
    # blocks that hold numbers next to the largest float (256 * 2^120), and blocks of the
    # smallest normal ones, as quantisation makes them
    import torch
    rng = np.random.default_rng(M)
    K = 384
    x, w = rng.standard_normal((M, K)), rng.standard_normal((N, K))
    x[:, :128] = np.finfo(np.float32).max * np.sign(x[:, :128])
    w[:, :128] *= 2.0 ** -120
    x[:, 128:256] *= 2.0 ** -122
    w[:, 128:256] *= 2.0 ** 110
    a, b = (lib.fp8_quantize(torch.from_numpy(t.astype(np.float32)).cuda()) for t in (x, w))
    va, vb = values(a), values(b)
    assert np.abs(va).max() == 2.0 ** 128
    got = host(lib.fp8_matmul(a, b, out_dtype=torch.float32))
    check_product(got[::M // 4], va[::M // 4], vb, "f32")


@pytest.mark.parametrize("M,N", [(4, 40), (1024, 1024)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scale_bytes_of_both_ends(lib, M, N, dtype):
    # byte 0 is 2^-127, byte 254 is 2^127, byte 255 is a NaN: its row and no other one
    import torch
    rng = np.random.default_rng(5)
    a, b = operand(lib, rng, M, 256, "e4m3")[0], operand(lib, rng, N, 256, "e5m2")[0]
    sa, sb = a.scale.view(torch.uint8), b.scale.view(torch.uint8)
    sa[:, 0], sb[:, 0] = 0, 238
    sa[1::2, 0], sa[:, 1], sb[:, 1] = 16, 254, 0
    va, vb = values(a), values(b)
    sa[2, 0], sb[3, 1] = 255, 255
    got = host(lib.fp8_matmul(a, b, out_dtype=torch.float32 if dtype == "f32" else torch.bfloat16))
    assert np.all(np.isnan(got[2])) and np.all(np.isnan(got[:, 3]))
    rows, cols = [0, 1, 3, M - 1], [c for c in range(N) if c != 3]
    # the same products of factors nearer to one
    near = np.repeat([2.0 ** 100, 2.0 ** -100], 128)
    check_product(got[np.ix_(rows, cols)], va[rows] * near, vb[cols] / near, dtype)


@pytest.mark.parametrize("M,N", [(4, 40), (1024, 1024)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_scale_of_zeros(lib, M, N, dtype):
    # 255 makes a block NaN whatever its values are
    import torch
    a, b = lib.fp8_quantize(torch.zeros(M, 256, device="cuda")), lib.fp8_quantize(torch.ones(N, 256, device="cuda"))
    a.scale.view(torch.uint8)[1, 1] = 255
    got = lib.fp8_matmul(a, b, out_dtype=torch.float32 if dtype == "f32" else torch.bfloat16)
    assert torch.all(torch.isnan(got[1]))
    got[1] = 0
    assert torch.all(got == 0)


@pytest.mark.parametrize("M,N,K", [(5, 40, 300), (1030, 1000, 600), (2100, 4000, 260)])
def test_results_that_are_not_finite(lib, M, N, K):
    # infinities and sums beyond the largest float, next to ordinary results of the same tile
    import torch
    rng = np.random.default_rng(M)
    x = rng.standard_normal((M, K)).astype(np.float32)
    x[1, 3], x[2, 5] = np.inf, -np.inf
    x[3] = 1e38 * (1 + rng.random(K))
    w = np.abs(rng.standard_normal((N, K))).astype(np.float32) + 0.5
    a, b = lib.fp8_quantize(torch.from_numpy(x).cuda(), "e5m2"), lib.fp8_quantize(torch.from_numpy(w).cuda())
    out = torch.full((M, N), 2.0, device="cuda")
    got = host(lib.fp8_matmul(a, b, out=out, accumulate=True))
    assert np.all(got[1] == np.inf) and np.all(got[2] == -np.inf) and np.all(got[3] == np.inf)
    rows = [0, 4, M - 1]
    check_product(got[rows], values(a)[rows], values(b), "f32", np.full((1, 1), 2.0))
