"""GPU: the columns behind an operand's last one hold zeros whatever the row's weight is."""
import numpy as np
import pytest

from oracle import fp8 as F
from test_gpu_fp8 import check_operand, dt, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("out,cols", [(5, 1), (40, 131), (130, 260), (300, 384)])
def test_infinite_and_nan_weights(lib, out, cols, dtype, fmt):
    import torch
    rng = np.random.default_rng([out, cols])
    x = torch.from_numpy(rng.standard_normal((out, cols)).astype(np.float32)).to(dt(torch, dtype)).cuda()
    w = rng.standard_normal(out).astype(np.float32)
    w[0], w[out // 2], w[-1] = np.nan, np.inf, -np.inf
    index = rng.permutation(out).astype(np.int32)
    index[1] = -1
    q, qt = lib.fp8_quantize(x, fmt, transposed="both", row_index=torch.from_numpy(index).cuda(),
                             row_weight=torch.from_numpy(w).cuda())
    with np.errstate(invalid="ignore"):
        g = F.gather(host(x), index, 1, w)
    check_operand(q, *F.quantize(g, fmt), out, cols)
    check_operand(qt, *F.quantize(g.T, fmt), cols, out)
