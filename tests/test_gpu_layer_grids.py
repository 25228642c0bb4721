"""GPU: norm, embedding and attention with more workgroups than one dimension of a grid is given
(2^20), and sorts of more tokens than one round of their blocks holds.

Bounds as in test_gpu_layer_ops; all references are elementwise in float64 on the GPU.
"""
import pytest

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF16 = 2.0 ** -8
MANY = 1 << 20   # workgroups


def normal(seed, *shape):
    import torch
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def test_norm_of_many_rows(lib):
    rows, cols = 4 * MANY + 4099, 8
    x, dy = normal(1, rows, cols), normal(2, rows, cols)
    n = lib.rms_norm(x)
    rstd = (x.double().square().mean(1) + 1e-6).rsqrt()
    want = x.double() * rstd[:, None]
    assert ((n.rstd.double() - rstd).abs() <= 30 * U * rstd).all()
    assert ((n.y.double() - want).abs() <= 32 * U * want.abs()).all()
    dx = lib.rms_norm_backward(dy, x, None, n.rstd)[0]
    g, r = dy.double(), n.rstd.double()[:, None]
    unit = x.double() * r
    want = r * (g - unit * (g * unit).mean(1, keepdim=True))
    size = r * (g.abs() + unit.abs() * (g * unit).abs().mean(1, keepdim=True))
    assert ((dx.double() - want).abs() <= 64 * U * size).all()


def test_embedding_of_many_tokens(lib):
    import torch
    tokens, vocab, cols = 4 * MANY + 77, 70001, 8
    table = normal(3, vocab, cols).bfloat16()
    ids = torch.randint(-1, vocab, (tokens,), generator=torch.Generator(device="cuda").manual_seed(4), device="cuda")
    y = lib.embedding(ids, table, scale=2.0)
    assert torch.equal(y, torch.where(ids[:, None] >= 0, 2.0 * table[ids.clamp(min=0)], 0.0))
    # whole numbers: every order of sums gives the same
    dy = torch.randint(-8, 9, (tokens, cols), generator=torch.Generator(device="cuda").manual_seed(5), device="cuda").float()
    want = torch.zeros(vocab + 1, cols, dtype=torch.float64, device="cuda").index_add_(0, torch.where(ids < 0, vocab, ids), dy.double())
    got = lib.embedding_backward(dy, ids, vocab)
    assert torch.equal(got.double(), want[:vocab])
    assert torch.equal(lib.embedding_backward(dy, ids, vocab, out=got.clone(), accumulate=True), 2 * got)


@pytest.mark.parametrize("tokens", [5000, 262145, 1000003])
def test_sorts_of_many_tokens(lib, tokens):
    """Blocks of 1024 tokens up to 256 of them, then longer ones; one id takes every third token."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(tokens)
    vocab, cols = 1 << 17, 24
    ids = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
    ids[::3] = vocab - 1
    dy = torch.randint(-8, 9, (tokens, cols), generator=g, device="cuda").to(torch.bfloat16)
    want = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda").index_add_(0, ids, dy.double())
    assert torch.equal(lib.embedding_backward(dy, ids, vocab).double(), want)


def test_gradient_of_a_table_of_many_rows(lib):
    import torch
    vocab, cols = 4 * MANY + 5, 3
    ids = torch.tensor([0, 7, vocab - 1, 4 * MANY, 7, vocab], device="cuda")
    dy = normal(6, 6, cols)
    want = torch.zeros(vocab, cols, device="cuda")
    want[0], want[7], want[vocab - 1], want[4 * MANY] = dy[0], dy[1] + dy[4], dy[2], dy[3]
    out = torch.full((vocab, cols), float("nan"), device="cuda")
    assert torch.equal(lib.embedding_backward(dy, ids, vocab, out=out), want)


@pytest.mark.parametrize("heads", [16, 15])
def test_attention_of_many_tiles(lib, heads):
    """A token by itself sees itself alone: out is its value, the log-sum-exp its score, dv the output's gradient."""
    import torch
    tokens, dim = 70001, 8
    assert tokens * heads > MANY
    q, k, v, do = (normal(7 + i, tokens, heads, dim).bfloat16() for i in range(4))
    off = torch.arange(tokens + 1, dtype=torch.int32, device="cuda")
    out, lse = lib.attention(q, k, v, offsets=off)
    assert torch.equal(out, v)
    score = (q.double() * k.double()).sum(2) * dim ** -0.5
    size = (q.double() * k.double()).abs().sum(2) * dim ** -0.5
    assert ((lse.t().double() - score).abs() <= 16 * U * (size + 1)).all()
    dq, dk, dv = lib.attention_backward(do, q, k, v, out, lse, offsets=off)
    assert torch.equal(dv, do)
    # dP and delta are the same sum in two orders: what is left is their rounding, and the probability's
    noise = 2 * (dim + 8) * U * (do.double() * v.double()).abs().sum(2, keepdim=True) * dim ** -0.5 * (1 + HALF16)
    assert (dq.double().abs() <= noise * k.double().abs() * (1 + HALF16) + 2.0 ** -126).all()
    assert (dk.double().abs() <= noise * q.double().abs() * (1 + HALF16) + 2.0 ** -126).all()
