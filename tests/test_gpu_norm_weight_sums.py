"""GPU: the norm's weight gradient where each workgroup's sum is exact.

Whole numbers with rstd 1: what a workgroup adds up (at most 22 rows of products below 700^2) is a whole
number below 2^24, exact in fp32. The workgroups' sums are joined in 64 bits and rounded once.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [9, 40, 2048, 2500])
@pytest.mark.parametrize("accumulate", [False, True])
def test_joined_sums_are_rounded_once(lib, cols, accumulate):
    import torch
    rows = 16384
    assert (rows // 768 + 1) * 699 ** 2 < 2 ** 24
    rng = np.random.default_rng(cols)
    s, dy = rng.integers(1, 700, (rows, cols)), rng.integers(-200, 700, (rows, cols))
    before = rng.integers(-9999, 9999, cols) if accumulate else np.zeros(cols, np.int64)
    want = (np.sum(s * dy, axis=0) + before).astype(np.float64)
    assert np.abs(want).max() > 2 ** 24
    dev = [torch.from_numpy(x.astype(np.float32)).cuda() for x in (s, dy, np.ones(rows), np.ones(cols), before)]
    dw = lib.rms_norm_backward(dev[1], dev[0], dev[3], dev[2], dweight=dev[4], accumulate=accumulate)[1]
    assert np.array_equal(dw.cpu().numpy(), want.astype(np.float32))
