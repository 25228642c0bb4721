"""GPU: the norm's 1 / rms where the sum over a row is exact.

Whole numbers up to 8: squares and sums of up to 16384 of them are whole numbers below 2^24, exact in
fp32 in any order. What is left is one rounding: the nearest float32 to (mean + eps)^(-1/2).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1, 7, 100, 1000, 2048, 4096, 11008, 16384])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-2])
def test_root_is_rounded_once(lib, cols, dtype, eps):
    import torch
    kind = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    rng = np.random.default_rng(cols)
    x = rng.integers(1, 9, (400, cols)) * rng.choice([-1, 1], (400, cols))
    x[100:200] //= 3   # rows of small numbers, some of them zeros
    x[100:200, 0] = 1
    total = np.sum(x * x, axis=1)
    assert total.max() < 2 ** 24
    got = lib.rms_norm(torch.from_numpy(x).to(kind).cuda(), eps=eps).rstd.cpu().numpy()
    want = (1 / np.sqrt(total / cols + float(np.float32(eps)))).astype(np.float32)
    assert np.array_equal(got, want)


def test_roots_at_the_ends(lib):
    import torch
    rows = torch.zeros(5, 300, device="cuda")
    rows[1] = 1e-20    # squares of 1e-40
    rows[2] = 1e19     # sums beyond fp32
    rows[3], rows[4] = float("inf"), float("nan")
    got = lib.rms_norm(rows, eps=0.0).rstd.double().cpu().numpy()
    assert got[0] == np.inf and abs(got[1] / 1e20 - 1) <= 2.0 ** -15 and got[2] == 0 and got[3] == 0 and np.isnan(got[4])
