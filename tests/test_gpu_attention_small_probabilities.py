"""GPU: many small probabilities next to a large one, in fp16.

Key 0 takes most of every row; each of the n others gets 2^-25.5 of it, which is less than fp16 holds,
while all of them together are a part of the result that fp16 shows clearly. The probabilities are
rounded to fp16 under 2^7 (forward, of the row's maximum) and 2^14 (gradient, of 1): below 2^-14 of
the scale that they carry they are off by 2^-25 of it, which is 2^-32 and 2^-39. In closed form all
rows are equal:
  p = e / (1 + n e) of the n keys and p0 = 1 / (1 + n e) of key 0, with e = exp(-d).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

HALF, U = 2.0 ** -11, 2.0 ** -24


def rows(tokens, first):
    """q, k, v of one head: the loud key is the first one or the last one; d, the distance of scores."""
    import torch
    q = torch.zeros(tokens, 1, 8, dtype=torch.float16, device="cuda")
    k, v = torch.zeros_like(q), torch.zeros_like(q)
    loud = 0 if first else tokens - 1
    q[:, 0, 0] = 4.0
    k[loud, 0, 0] = 4.421875
    v[:, 0, 0] = 1.0
    v[loud, 0, 0], v[loud, 0, 1] = 0.0, 1.0
    return q, k, v, loud, 4.0 * 4.421875


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("tokens", [8192, 70001])
def test_small_probabilities_add_up(lib, tokens, first):
    import torch
    q, k, v, loud, d = rows(tokens, first)
    n, e = tokens - 1, np.exp(-d)
    assert 2.0 ** -26 < e < 2.0 ** -25
    total = 1 + n * e
    p, p0 = e / total, 1 / total
    out, lse = lib.attention(q, k, v, causal=False, scale=1.0)
    out, lse_host = out.double().cpu().numpy()[:, 0], lse.double().cpu().numpy()[0]
    # half a step of the probability and of the result; sums of n; the exponential's own error
    off = 2 * HALF + 2 * U * (n + 64)
    for column, want in ((0, n * p), (1, p0)):
        assert np.all(np.abs(out[:, column] - want) <= off * want + n * 2.0 ** -32 + 2.0 ** -24), column
    assert np.all(np.abs(lse_host - (d + np.log(total))) <= U * (n + 64))
    do = torch.zeros_like(q)
    do[:, 0, 0] = 1.0
    o = torch.zeros_like(q)
    o[:, 0, 0] = n * p
    dv = lib.attention_backward(do, q, k, v, o, lse, causal=False, scale=1.0)[2].double().cpu().numpy()[:, 0, 0]
    others = np.arange(tokens) != loud
    assert np.all(np.abs(dv[others] - tokens * p) <= off * tokens * p + tokens * 2.0 ** -39 + 2.0 ** -24)
    # the loud key's is about the number of rows, which fp16 holds to 65504
    if tokens < 65000:
        assert abs(dv[loud] - tokens * p0) <= off * tokens * p0
