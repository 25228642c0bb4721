"""GPU: clipping by factors below fp32's smallest normal number.

The factor keeps 24 bits down to where every result is 0: a result is two fp32 products and the
roundings of the factor and of the output's type off, and half of the smallest number of its type
where it leaves the normal ones.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
LOW = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133}
U = 2.0 ** -24


@pytest.mark.parametrize("out", [None, "f32", "bf16"])
@pytest.mark.parametrize("size,max_norm", [(1e9, 1e-30), (3e38, 1e-3), (3e38, 1e-8), (1e38, 1e-44), (1.0, 1e-37), (1.0, 1e-39)])
def test_small_factors(lib, size, max_norm, out):
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    grads = [(torch.rand(n, generator=g, device="cuda") * 2 - 1) * size for n in (8193, 77, 20000)]
    grads[1] *= 1e-30
    values = [t.double().cpu().numpy() for t in grads]
    exact = np.sqrt(sum(float(np.sum(v * v)) for v in values))
    max_norm = float(np.float32(max_norm))
    factor = max_norm / (exact + 1e-6)
    assert factor < 2.0 ** -126
    kind = {None: None, "f32": torch.float32, "bf16": torch.bfloat16}[out]
    outs = None if kind is None else [torch.full_like(t, float("nan"), dtype=kind) for t in grads]
    norm = lib.clip_gradients(grads, max_norm, out=outs)
    with np.errstate(over="ignore"):
        assert norm.item() == pytest.approx(float(np.float32(exact)), rel=2 * U)
    name = out or "f32"
    for t, v in zip(outs or grads, values):
        got, want = t.double().cpu().numpy(), v * factor
        assert np.all(np.abs(got - want) <= (HALF[name] + 4 * U) * np.abs(want) + 2 * LOW[name])
