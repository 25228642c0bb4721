"""GPU: group offsets that fall. One that is less than an earlier one counts as the largest
before it: no row and no column belongs to two groups, on every kernel and with more groups
than a wave looks at together. Tolerances as in test_gpu_fp8.py."""
import numpy as np
import pytest

from test_gpu_fp8 import check_product, dt, host, kinds, operand

pytestmark = pytest.mark.gpu


def spans(off, limit):
    """Rows (or columns) of each group."""
    o = np.maximum.accumulate(np.clip(np.asarray(off, np.int64), 0, limit))
    return list(zip(o[:-1], o[1:]))


def falling(rng, groups, limit, align=1):
    """Offsets that rise on the whole and fall every now and then, far beyond the limit too."""
    off = np.sort(rng.integers(0, limit // align + 1, groups + 1)) * align
    at = rng.permutation(groups)[:max(2, groups // 4)] + 1
    off[at] = rng.integers(-2, limit // align // 2, len(at)) * align
    if groups > 10:
        off[groups // 2] = 0
        off[-2] = 2 ** 31 - align
    return off


def of_few(lib, rng, groups, rows, cols):
    """`groups` matrices, five different ones in turn, and their values."""
    op, v = operand(lib, rng, rows, cols, "e4m3", 5)
    turn = [g % 5 for g in range(groups)]
    import torch
    data = op.data.view(torch.uint8)[turn].view(op.data.dtype)
    scale = op.scale.view(torch.uint8)[turn].view(op.scale.dtype)
    return lib.Fp8(data, scale, cols), [v[t] for t in turn]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K,G,kernel", [(200, 40, 200, 3, "few_rows"), (200, 40, 200, 70, "few_rows"),
                                            (1500, 1300, 520, 7, "128"), (1500, 1300, 520, 140, "128"),
                                            (9000, 3000, 136, 75, "256")])
def test_rows(lib, M, N, K, G, kernel, dtype):
    import torch
    rng = np.random.default_rng([M, G])
    a, va = operand(lib, rng, M, K, "e4m3")
    b, vb = of_few(lib, rng, G, N, K)
    for off in (falling(rng, G, M), [M // 4, M // 2, M // 5] + [M] * (G - 2)):
        offsets = torch.from_numpy(np.asarray(off).astype(np.int32)).cuda()
        out = torch.full((M, N), 0.5, dtype=dt(torch, dtype), device="cuda")
        ran = kinds(lib, lambda: lib.fp8_matmul(a, b, out=out, offsets=offsets, accumulate=True))
        assert ran == {"fp8_gemm_" + kernel}
        cols = rng.permutation(N)[:40]
        got = host(out[:, torch.from_numpy(cols).cuda()])
        owned = np.zeros(M, bool)
        for g, (lo, hi) in enumerate(spans(off, M)):
            check_product(got[lo:hi], va[lo:hi], vb[g][cols], dtype, np.full((1, 1), 0.5))
            owned[lo:hi] = True
        assert torch.all(out[torch.from_numpy(~owned).cuda()] == 0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,blocks,G,kernel", [(20, 40, 9, 5, "few_rows"), (20, 40, 9, 70, "few_rows"),
                                                 (300, 260, 100, 70, "128"), (512, 512, 37, 4, "128"),
                                                 (1024, 1000, 30, 70, "256")])
def test_contractions(lib, M, N, blocks, G, kernel, dtype):
    import torch
    rng = np.random.default_rng([M, G])
    a, va = operand(lib, rng, M, 128 * blocks, "e5m2")
    b, vb = operand(lib, rng, N, 128 * blocks, "e4m3")
    for off in (falling(rng, G, 128 * blocks, 128), [128 * 2, 128 * 5, 128] + [128 * blocks] * (G - 2)):
        offsets = torch.from_numpy(np.asarray(off).astype(np.int32)).cuda()
        out = torch.full((G, M, N), 7.0, dtype=dt(torch, dtype), device="cuda")
        ran = kinds(lib, lambda: lib.fp8_matmul_grouped_k(a, b, offsets, out=out))
        assert ran == {"fp8_gemm_" + kernel}
        rows = np.arange(0, M, max(1, M // 12))
        got = host(out[:, torch.from_numpy(rows).cuda()])
        for g, (lo, hi) in enumerate(spans(off, 128 * blocks)):
            check_product(got[g], va[rows, lo:hi], vb[:, lo:hi], dtype)
