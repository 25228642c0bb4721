"""GPU: the log-sum-exp of rows that see one key, whose scores are exact in fp32.

It is the score itself. An exponential next to a power of two is off by one step of fp32 (2 U), its
logarithm as much, and the sum with the scaled score is rounded once (U of it).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [8, 64, 128])
def test_one_key(lib, dim, dtype):
    import torch
    kind = {"bf16": torch.bfloat16, "f16": torch.float16}[dtype]
    tokens = 3000
    g = torch.Generator(device="cuda").manual_seed(dim)
    q, k = (torch.zeros(tokens, 2, dim, device="cuda") for _ in range(2))
    q[..., :2] = torch.randint(-127, 128, (tokens, 2, 2), generator=g, device="cuda") / 16
    k[..., :2] = torch.randint(-127, 128, (tokens, 2, 2), generator=g, device="cuda") / 64
    q, k = q.to(kind), k.to(kind)
    score = (q.double() * k.double()).sum(2) / 4
    off = torch.arange(tokens + 1, dtype=torch.int32, device="cuda")
    lse = lib.attention(q, k, k, offsets=off, scale=0.25)[1].t().double()
    off = (lse - score).abs()
    assert (off <= 3 * U + U * score.abs()).all(), (off / (3 * U + U * score.abs())).max()
