"""GPU: calls whose kernels need more than 2^32 threads, more than one dimension of a grid
takes. Every element behind the border is checked, by exact values where there are some."""
import pytest

pytestmark = pytest.mark.gpu


def test_route_and_its_gradient_of_many_tokens(lib):
    import torch
    tokens = (1 << 26) + 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randint(-8, 9, (tokens, 2), device="cuda", generator=gen, dtype=torch.int8).to(torch.bfloat16)
    ids = torch.full((tokens, 1), 7, dtype=torch.int32, device="cuda")
    weights = torch.full((tokens, 1), 7.0, device="cuda")
    lib.route(logits, lib.route_hyper(top_k=1), ids=ids, weights=weights)
    assert torch.equal(ids[:, 0], (logits[:, 1] > logits[:, 0]).int())
    assert torch.all(weights == 1.0)      # s / (s + 1e-20), s >= 1 / 2
    # without renormalisation the weight is s_c and its gradient s_c (1 - s_c), and its
    # negative for the other one; s_c (1 - s_c) >= e^-16 / 2, rounded once to fp32, once to bf16
    dlogits = torch.full_like(logits, 7.0)
    lib.route_backward(torch.ones_like(weights), logits, ids, lib.route_hyper(top_k=1, renormalize=0), dlogits=dlogits)
    for part in (slice(0, 1 << 20), slice(tokens - (1 << 20), tokens)):
        l = logits[part].double()
        s = torch.sigmoid((l[:, 0] - l[:, 1]).abs())
        want = s * torch.sigmoid(-(l[:, 0] - l[:, 1]).abs())
        d = dlogits[part].double()
        first = ids[part, 0] == 0
        sign = torch.where(first, 1.0, -1.0).double()
        tol = (2.0 ** -8 + 2.0 ** -20) * want
        assert torch.all((d[:, 0] - sign * want).abs() <= tol)
        assert torch.all((d[:, 1] + sign * want).abs() <= tol)
    assert not torch.any(dlogits == 7.0)


def test_combine_and_its_gradient_of_many_tokens(lib):
    import torch
    tokens, cols = (1 << 24) + 5, 8
    o = torch.arange(3 * cols, device="cuda").view(3, cols).to(torch.bfloat16)
    t = torch.arange(tokens, device="cuda")
    pos = (t % 5 - 1).int().view(-1, 1)                       # -1 and 3: no row
    w = (2.0 ** (t % 3).float()).view(-1, 1)
    y = torch.full((tokens, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.combine(o, pos, w, out=y)
    has = (pos >= 0) & (pos < 3)
    rows = torch.where(has, pos, 0).long()[:, 0]
    want = torch.where(has, o[rows] * w.to(torch.bfloat16), 0)   # small integers: exact
    assert torch.equal(y, want)
    # the gradient: every token but the last three points at no row, so that no two share one
    pos = torch.full((tokens, 1), -1, dtype=torch.int32, device="cuda")
    pos[-3:, 0] = torch.arange(3, device="cuda").int()
    dw = torch.full((tokens, 1), 7.0, device="cuda")
    do = torch.full_like(o, 7.0)
    dy = torch.ones((tokens, cols), dtype=torch.bfloat16, device="cuda")
    lib.combine_backward(dy, o, pos, w, dweights=dw, do=do)
    assert torch.all(dw[:-3] == 0)
    assert torch.equal(dw[-3:, 0], o.float().sum(1))
    assert torch.equal(do, w[-3:].to(torch.bfloat16).expand(3, cols))


def test_quantize_many_tiles(lib):
    import torch
    batch, rows = 1024, (1 << 21) + 200
    x = torch.randn((rows, 1), device="cuda").to(torch.bfloat16)
    one = lib.fp8_quantize(x, transposed="only")
    many = lib.fp8_quantize(x.expand(batch, rows, 1), transposed="only")
    want, want_s = one.data.view(torch.uint8), one.scale.view(torch.uint8)
    got, got_s = many.data.view(torch.uint8), many.scale.view(torch.uint8)
    for i in range(batch):
        assert torch.equal(got[i], want), i
        assert torch.equal(got_s[i], want_s), i


def test_few_rows_many_workgroups(lib):
    import torch
    n, groups = 1 << 22, 40
    x = torch.randint(-3, 4, (n, 128), device="cuda", dtype=torch.int8).float()
    a = torch.randint(-3, 4, (1, 128), device="cuda", dtype=torch.int8).float()
    b8, a8 = lib.fp8_quantize(x), lib.fp8_quantize(a)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = 128
    out = torch.full((groups, 1, n), 7.0, device="cuda")
    lib.profile_begin()
    lib.fp8_matmul_grouped_k(a8, b8, offsets, out=out)
    assert set(lib.profile_end()) == {"fp8_gemm_few_rows"}
    assert torch.equal(out[-1, 0], (x * a).sum(1))    # small integers: exact
    assert torch.all(out[:-1] == 0)
