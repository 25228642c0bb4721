"""GPU: 8-bit operands and their products against the float64 oracle.

Quantisation has to give the oracle's values and scales exactly (both round the same
exact number once). A product's terms are exact in fp32 (8-bit times 8-bit times powers
of two), so its error comes from at most K + 16 additions, each off by at most 2^-23 of
the running magnitude (a whole unit: the rounding inside the matrix instruction is not
documented), and one final rounding of half a step of the result's type:
  |c - exact| <= (K + 16) 2^-23 sum |a b| + half |exact| (1 + small)
A 16-bit result comes from the 8-bit matrix instructions. They add eight neighbouring
products along k at a time, each cut to a multiple of 2^-13 times the power of two at or
below the largest of the eight (seen in the instruction itself: beside 2^e a product of
2^(e - 13) is kept and the part below is dropped; a product more than seven places away
is kept whole). So each of the other seven loses less than 2^-13 of the largest product,
and the largest nothing:
  |c - exact| <= ... + 7 * 2^-13 sum over eights of max |a b|
"""
import numpy as np
import pytest

from oracle import fp8 as F

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


def dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def host(t):
    return t.detach().float().cpu().double().numpy()


def check_operand(op, want_q, want_e, rows, cols):
    """data and scale of an Fp8 against the oracle's, padding included."""
    import torch
    q = op.data.detach().cpu().float().double().numpy()
    assert q.shape == want_q.shape
    assert np.array_equal(q, want_q, equal_nan=True)
    e = op.scale.detach().cpu().view(torch.uint8).numpy().astype(np.int64) - 127
    nb = want_e.shape[1]
    assert np.array_equal(e[:, :nb], want_e)
    assert np.all(e[:, nb:] == 0)
    assert e.shape[1] == F.up(nb, 4)


def source(rng, rows, cols, kind="normal"):
    x = rng.standard_normal((rows, cols)) * np.exp(rng.standard_normal(cols))
    if kind == "wide" and x.size:       # tiny, huge and zero blocks, values on the borders of the scale rule
        x *= 10.0 ** rng.integers(-30, 30, (rows, 1))
        x[rng.random((rows, cols)) < 0.3] = 0.0
        x[::5] = 0.0
        x[0, 0], x[-1, -1] = 448.0, 57344.0
    return x


@pytest.mark.parametrize("blocks", [False, True])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 130), (128, 128), (129, 127), (200, 515), (1, 1000), (700, 8)])
def test_quantize(lib, rows, cols, dtype, fmt, blocks):
    import torch
    rng = np.random.default_rng([rows, cols, len(fmt), blocks])
    for kind in ("normal", "wide") if dtype == "f32" else ("normal",):
        x = torch.from_numpy(source(rng, rows, cols, kind).astype(np.float32)).to(dt(torch, dtype)).cuda()
        q, qt = lib.fp8_quantize(x, fmt, blocks=blocks, transposed="both")
        only = lib.fp8_quantize(x, fmt, blocks=blocks)
        only_t = lib.fp8_quantize(x, fmt, blocks=blocks, transposed="only")
        torch.cuda.synchronize()
        xs = host(x)
        want, want_t = F.quantize(xs, fmt, blocks), F.quantize(xs.T, fmt, blocks)
        for op in (q, only):
            check_operand(op, *want, rows, cols)
        for op in (qt, only_t):
            check_operand(op, *want_t, cols, rows)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_non_finite_and_borders(lib, fmt):
    # a NaN or an infinity stays one and leaves its block's scale alone; amax at and just
    # beyond 1.75 * 2^k; subnormals; the largest float
    import torch
    x = np.zeros((8, 256), np.float32)
    x[0, :4] = [np.nan, 1.0, -2.0, 0.5]
    x[1, :4] = [np.inf, -np.inf, 3.0, 1e-3]
    x[2, 0] = 1.75
    x[3, 0] = np.nextafter(np.float32(1.75), np.float32(2))
    x[4, :3] = [1e-45, 1e-40, 3e-39]
    x[5, :2] = [np.finfo(np.float32).max, -1.0]
    x[6, 128:] = np.nan
    x[7] = np.linspace(-3, 3, 256)
    t = torch.from_numpy(x).cuda()
    q, qt = lib.fp8_quantize(t, fmt, transposed="both")
    torch.cuda.synchronize()
    check_operand(q, *F.quantize(x.astype(np.float64), fmt), 8, 256)
    check_operand(qt, *F.quantize(x.T.astype(np.float64), fmt), 256, 8)


def test_quantize_rounds_ties_to_even(lib):
    import torch
    # every midpoint of neighbouring e4m3 values below 448, and its two neighbours, beside
    # an amax of 448 that fixes the scale at 1
    vals = np.unique(np.abs(F.decode_table("e4m3")[np.isfinite(F.decode_table("e4m3"))]))
    mid = (vals[1:] + vals[:-1]) / 2
    cand = np.concatenate([mid, np.nextafter(mid.astype(np.float32), np.float32(1e9)),
                           np.nextafter(mid.astype(np.float32), np.float32(0))]).astype(np.float32)
    rows = -(-len(cand) // 127)
    x = np.zeros((rows, 128), np.float32)
    x[:, 0] = 448.0
    x[:, 1:].flat[:len(cand)] = cand
    q = lib.fp8_quantize(torch.from_numpy(x).cuda(), "e4m3")
    torch.cuda.synchronize()
    check_operand(q, *F.quantize(x.astype(np.float64), "e4m3"), rows, 128)


@pytest.mark.parametrize("div,weighted", [(1, False), (6, False), (3, True)])
def test_quantize_gathers_rows(lib, div, weighted):
    import torch
    rng = np.random.default_rng(div)
    rows, cols, out = 50, 300, 333
    x = torch.from_numpy(source(rng, rows, cols).astype(np.float32)).bfloat16().cuda()
    n = rows * div
    index = rng.integers(0, n, out).astype(np.int32)
    index[::7] = -1
    index[5], index[6], index[8] = n, 2 ** 31 - 1, -2 ** 31      # beyond the source: zeros
    w = rng.standard_normal(n - 3).astype(np.float32) if weighted else None   # the last slots have no weight
    q, qt = lib.fp8_quantize(x, "e4m3", transposed="both", row_index=torch.from_numpy(index).cuda(), row_div=div,
                             row_weight=None if w is None else torch.from_numpy(w).cuda())
    torch.cuda.synchronize()
    g = F.gather(host(x), index, div, w)
    check_operand(q, *F.quantize(g, "e4m3"), out, cols)
    check_operand(qt, *F.quantize(g.T, "e4m3"), cols, out)


def test_quantize_reads_views(lib):
    # matrices inside a packed buffer: a batch with its own stride, odd offsets and pitches
    import torch
    rng = np.random.default_rng(9)
    buf = torch.from_numpy(rng.standard_normal(4 * 40 * 210 + 11).astype(np.float32)).cuda()
    before = buf.clone()
    for off, pitch, cols in ((0, 208, 208), (3, 205, 200), (8, 200, 131), (0, 0, 77)):
        v = buf[off:].as_strided((3, 37, cols), (41 * 205, pitch, 1))
        q, qt = lib.fp8_quantize(v, "e5m2", blocks=True, transposed="both")
        torch.cuda.synchronize()
        xs = host(v)
        for i in range(3):
            w, wt = F.quantize(xs[i], "e5m2", True), F.quantize(xs[i].T, "e5m2", True)
            check_operand(lib.Fp8(q.data[i], q.scale[i], q.cols), *w, 37, cols)
            check_operand(lib.Fp8(qt.data[i], qt.scale[i], qt.cols), *wt, cols, 37)
    assert torch.equal(buf, before)


# ----------------------------------------------------------------------------- products

def operand(lib, rng, rows, cols, fmt, batch=None):
    """A quantised operand on the GPU and its exact values."""
    import torch
    lead = () if batch is None else (batch,)
    x = rng.standard_normal(lead + (rows, cols)) * np.exp(0.5 * rng.standard_normal(cols))
    x *= 2.0 ** rng.integers(-6, 6, lead + (rows, 1))
    op = lib.fp8_quantize(torch.from_numpy(x.astype(np.float32)).cuda(), fmt)
    return op, values(op)


def values(op):
    q = host(op.data)
    e = op.scale.cpu().view(__import__("torch").uint8).numpy().astype(np.int64) - 127
    flat = F.dequantize(q.reshape(-1, q.shape[-1]), e.reshape(-1, e.shape[-1])[:, :q.shape[-1] // 128], op.cols)
    return flat.reshape(q.shape[:-1] + (op.cols,))


def eights(va, vb):
    """Sum over the groups of eight neighbours along k of the largest |a b| of each."""
    a, b = np.abs(va).astype(np.float32), np.abs(vb).astype(np.float32)
    out = np.zeros((a.shape[0], b.shape[0]))
    for k in range(0, a.shape[1], 8):
        most = np.zeros(out.shape, np.float32)
        for i in range(k, min(k + 8, a.shape[1])):
            np.maximum(most, a[:, i:i + 1] * b[:, i], out=most)
        out += most
    return out


def check_product(got, va, vb, dtype, base=None):
    """Against the bound of the module's docstring."""
    exact = va @ vb.T
    mag = np.abs(va) @ np.abs(vb).T
    if base is not None:
        exact = exact + base
        mag = mag + np.abs(base)
    K = va.shape[1]
    tol = (K + 16) * 2.0 ** -23 * mag
    if dtype != "f32":
        tol = tol + 7 * 2.0 ** -13 * eights(va, vb)
    tol = tol + HALF[dtype] * (np.abs(exact) + tol) + TINY[dtype]
    assert np.all(np.abs(got - exact) <= tol), np.max(np.abs(got - exact) / (tol + 1e-300))


SHAPES = [(1, 1, 1), (1, 64, 128), (1, 300, 4096), (2, 17, 130), (16, 16, 512), (17, 33, 1000), (48, 500, 640),
          (100, 128, 1), (128, 128, 128), (130, 257, 260), (256, 256, 1024), (300, 515, 384), (513, 1, 700),
          (640, 768, 896)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(lib, M, N, K, dtype):
    import torch
    rng = np.random.default_rng([M, N, K])
    fa, fb = [("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")][(M + N + K) % 4]
    a, va = operand(lib, rng, M, K, fa)
    b, vb = operand(lib, rng, N, K, fb)
    s = 2.0 ** -10 if dtype == "f16" else 1.0      # keep fp16 results in range
    if dtype == "f16":
        a = lib.fp8_quantize(torch.from_numpy((va * s).astype(np.float32)).cuda(), fa)
        va = values(a)
    c = lib.fp8_matmul(a, b, out_dtype=dt(torch, dtype))
    torch.cuda.synchronize()
    check_product(host(c), va, vb, dtype)


@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
@pytest.mark.parametrize("fb", ["e4m3", "e5m2"])
@pytest.mark.parametrize("M,N,K", [(5, 40, 300), (200, 140, 300), (512, 512, 768)])
def test_product_formats_and_scale_bytes(lib, M, N, K, fa, fb):
    # scales that differ from block to block by up to 2^40, each block's own byte used
    import torch
    rng = np.random.default_rng([7, M])

    def make(rows, fmt):
        x = rng.standard_normal((rows, K))
        for k in range(0, K, 128):
            x[:, k:k + 128] *= 2.0 ** rng.integers(-20, 20, (rows, 1))
        op = lib.fp8_quantize(torch.from_numpy(x.astype(np.float32)).cuda(), fmt)
        return op, values(op)
    a, va = make(M, fa)
    b, vb = make(N, fb)
    c = lib.fp8_matmul(a, b, out_dtype=torch.float32)
    torch.cuda.synchronize()
    check_product(host(c), va, vb, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(3, 50, 256), (140, 129, 384), (512, 256, 256)])
def test_product_into_a_view_and_accumulate(lib, M, N, K, dtype):
    # a matrix of a packed gradient buffer at an odd offset with its own pitch; the rest
    # of the buffer stays as it was
    import torch
    rng = np.random.default_rng([M, K])
    a, va = operand(lib, rng, M, K, "e4m3")
    b, vb = operand(lib, rng, N, K, "e4m3")
    for off, pitch in ((0, N), (5, N + 3), (8, -(-N // 8) * 8 + 8)):
        buf = torch.from_numpy(rng.standard_normal(off + M * pitch + 9).astype(np.float32)).to(dt(torch, dtype)).cuda()
        before = buf.clone()
        v = buf[off:].as_strided((M, N), (pitch, 1))
        base = host(v)
        lib.fp8_matmul(a, b, out=v, accumulate=True)
        torch.cuda.synchronize()
        check_product(host(v), va, vb, dtype, base)
        first = host(v)
        lib.fp8_matmul(a, b, out=v)
        torch.cuda.synchronize()
        check_product(host(v), va, vb, dtype)
        assert not np.array_equal(first, host(v))
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask.as_strided((M, N), (pitch, 1), off).fill_(False)
        assert torch.equal(buf[mask], before[mask])


def test_product_batch(lib):
    import torch
    rng = np.random.default_rng(3)
    for B, M, N, K in ((3, 5, 70, 300), (4, 150, 140, 256), (5, 256, 256, 128)):
        a, va = operand(lib, rng, M, K, "e4m3", B)
        b, vb = operand(lib, rng, N, K, "e5m2", B)
        c = lib.fp8_matmul(a, b, out_dtype=torch.float32)
        torch.cuda.synchronize()
        for i in range(B):
            check_product(host(c[i]), va[i], vb[i], "f32")


def test_product_without_terms_or_rows(lib):
    import torch
    a, b = lib.fp8_empty(5, 0), lib.fp8_empty(7, 0)
    c = lib.fp8_matmul(a, b, out=torch.full((5, 7), 3.0, device="cuda"))
    assert torch.equal(c, torch.zeros(5, 7, device="cuda"))
    assert lib.fp8_matmul(lib.fp8_empty(0, 256), lib.fp8_empty(7, 256)).shape == (0, 7)
    q, qt = lib.fp8_quantize(torch.empty(0, 40, device="cuda"), transposed="both")
    assert q.data.shape == (0, 128) and qt.data.shape == (40, 0)


def test_product_nan_and_inf_stay_in_their_rows(lib):
    import torch
    rng = np.random.default_rng(1)
    for M, N, K in ((20, 40, 256), (256, 256, 256)):
        x = rng.standard_normal((M, K)).astype(np.float32)
        x[3, 7] = np.nan
        x[11, 200] = np.inf
        a = lib.fp8_quantize(torch.from_numpy(x).cuda(), "e5m2")
        b, vb = operand(lib, rng, N, K, "e4m3")
        c = host(lib.fp8_matmul(a, b, out_dtype=torch.float32))
        assert np.all(np.isnan(c[3])) and not np.any(np.isfinite(c[11]))
        keep = [i for i in range(M) if i not in (3, 11)]
        check_product(c[keep], values(a)[keep], vb, "f32")


GROUPS = [[0, 0, 0], [1, 0, 3], [16, 17, 0, 31, 1], [200, 0, 129, 5, 128, 0], [1] * 70, [0] * 65 + [300, 7]]


@pytest.mark.parametrize("counts", GROUPS)
@pytest.mark.parametrize("N,K,dtype", [(40, 200, "f32"), (260, 512, "bf16")])
def test_grouped_rows(lib, counts, N, K, dtype):
    # ragged groups, empty ones among them, rows before and behind all groups left alone
    import torch
    rng = np.random.default_rng([len(counts), N])
    G, lead, tail = len(counts), 3, 21
    off = lead + np.concatenate([[0], np.cumsum(counts)])
    M = int(off[-1]) + tail
    a, va = operand(lib, rng, M, K, "e4m3")
    b, vb = operand(lib, rng, N, K, "e4m3", G)
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    out = torch.full((M, N), 7.0, dtype=dt(torch, dtype), device="cuda")
    lib.fp8_matmul(a, b, out=out, offsets=offsets)
    torch.cuda.synchronize()
    got = host(out)
    assert np.all(got[:lead] == 7.0) and np.all(got[off[-1]:] == 7.0)
    for g in range(G):
        check_product(got[off[g]:off[g + 1]], va[off[g]:off[g + 1]], vb[g], dtype)
    out.fill_(0.5)
    lib.fp8_matmul(a, b, out=out, offsets=offsets, accumulate=True)
    got = host(out)
    for g in range(G):
        check_product(got[off[g]:off[g + 1]], va[off[g]:off[g + 1]], vb[g], dtype, np.full((1, 1), 0.5))


def test_grouped_rows_clamps_offsets(lib):
    # offsets beyond the matrix give the rows that are there, nothing outside is touched
    import torch
    rng = np.random.default_rng(5)
    a, va = operand(lib, rng, 50, 128, "e4m3")
    b, vb = operand(lib, rng, 20, 128, "e4m3", 3)
    guard = torch.full((60, 20), 7.0, device="cuda")
    for off, rows in (([-5, 10, 10, 5000], [(0, 10), (10, 10), (10, 50)]),
                      ([2 ** 30, 2 ** 30, 2 ** 30, 2 ** 31 - 1], [(50, 50)] * 3)):
        guard.fill_(7.0)
        lib.fp8_matmul(a, b, out=guard[:50], offsets=torch.tensor(off, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        got = host(guard)
        assert np.all(got[50:] == 7.0)
        for g, (lo, hi) in enumerate(rows):
            check_product(got[lo:hi], va[lo:hi], vb[g], "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(20, 40), (260, 300)])
def test_grouped_contraction(lib, M, N, dtype):
    import torch
    rng = np.random.default_rng([M])
    blocks = [0, 1, 3, 0, 2, 5, 0]
    off = 128 * np.concatenate([[0], np.cumsum(blocks)])
    K = int(off[-1]) + 300
    a, va = operand(lib, rng, M, K, "e5m2")
    b, vb = operand(lib, rng, N, K, "e4m3")
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    G = len(blocks)
    buf = torch.full((G, 2, M, N), 7.0, dtype=dt(torch, dtype), device="cuda")   # every second matrix of a stack
    out = buf[:, 1]
    lib.fp8_matmul_grouped_k(a, b, offsets, out=out)
    torch.cuda.synchronize()
    got = host(out)
    assert torch.all(buf[:, 0] == 7.0)
    for g in range(G):
        check_product(got[g], va[:, off[g]:off[g + 1]], vb[:, off[g]:off[g + 1]], dtype)
    out.fill_(0.25)
    lib.fp8_matmul_grouped_k(a, b, offsets, out=out, accumulate=True)
    got = host(out)
    for g in range(G):
        check_product(got[g], va[:, off[g]:off[g + 1]], vb[:, off[g]:off[g + 1]], dtype, np.full((1, 1), 0.25))


def test_product_gradients_by_differences(lib):
    # the three products of a layer agree: with y = x w^T and L = <dy, y>, the input and
    # weight gradients from transposed operands equal dy w and dy^T x, and moving a weight
    # moves L by its gradient
    import torch
    rng = np.random.default_rng(11)
    T, N, K = 200, 150, 270
    x = torch.from_numpy(rng.standard_normal((T, K)).astype(np.float32)).cuda()
    w = torch.from_numpy(rng.standard_normal((N, K)).astype(np.float32)).cuda()
    dy = torch.from_numpy(rng.standard_normal((T, N)).astype(np.float32)).cuda()
    xq, xt = lib.fp8_quantize(x, transposed="both")
    wq, wt = lib.fp8_quantize(w, blocks=True, transposed="both")
    dq, dtq = lib.fp8_quantize(dy, "e5m2", transposed="both")
    assert np.array_equal(values(wq), values(wt).T)
    y = host(lib.fp8_matmul(xq, wq, out_dtype=torch.float32))
    dx = host(lib.fp8_matmul(dq, wt, out_dtype=torch.float32))
    dw = host(lib.fp8_matmul(dtq, xt, out_dtype=torch.float32))
    check_product(y, values(xq), values(wq), "f32")
    check_product(dx, values(dq), values(wt), "f32")
    check_product(dw, values(dtq), values(xt), "f32")
    # the loss is linear in each weight: differences of the float64 loss over the values
    # the weight gradient's operands hold
    vd, vx = values(dtq).T, values(xt).T
    for n, k in ((0, 0), (149, 269), (77, 130)):
        v = values(wq)
        lo = (vd * (vx @ v.T)).sum()
        v[n, k] += 1.0
        hi = (vd * (vx @ v.T)).sum()
        mag = (np.abs(vd[:, n]) * np.abs(vx[:, k])).sum()
        assert abs((hi - lo) - dw[n, k]) <= (T + 16) * 2.0 ** -23 * mag + 1e-9 * (abs(hi) + abs(lo))


# products large enough for the widest tiles: many matrices, ragged groups and
# contractions, in every mode, both kinds of result; the launch statistics say which
# kernel ran

def kinds(lib, call):
    lib.profile_begin()
    call()
    return set(lib.profile_end())


def test_every_kernel_is_reached(lib):
    import torch
    for (m, n, k), want in (((1, 512, 512), "fp8_gemm_few_rows"), ((64, 512, 512), "fp8_gemm_few_rows"),
                            ((1024, 1024, 4096), "fp8_gemm_128"), ((4096, 4096, 256), "fp8_gemm_256")):
        a = lib.fp8_quantize(torch.zeros(m, k, device="cuda"))
        b = lib.fp8_quantize(torch.zeros(n, k, device="cuda"))
        for dtype in (torch.float32, torch.bfloat16):
            assert kinds(lib, lambda: lib.fp8_matmul(a, b, out_dtype=dtype)) == {want}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", [(500, 490, 300), (512, 512, 128), (257, 511, 1), (300, 260, 2100)])
def test_many_wide_tiles_batch(lib, M, N, K, dtype):
    import torch
    rng = np.random.default_rng([M, N])
    B = 64
    a, va = operand(lib, rng, M, K, "e4m3", B)
    b, vb = operand(lib, rng, N, K, "e5m2", B)
    buf = torch.full((B, M + 1, N + 3), 7.0, dtype=dt(torch, dtype), device="cuda")
    out = buf[:, :M, 3:]
    for acc in (False, True):
        base = host(out) if acc else None
        ran = kinds(lib, lambda: lib.fp8_matmul(a, b, out=out, accumulate=acc))
        assert M < 500 or ran == {"fp8_gemm_256"}
        torch.cuda.synchronize()
        got = host(out)
        for i in range(0, B, 13):
            check_product(got[i], va[i], vb[i], dtype, None if base is None else base[i])
    assert torch.all(buf[:, M] == 7.0) and torch.all(buf[:, :, :3] == 7.0)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("counts", [[0, 700, 1, 0, 255, 257, 256, 0, 40, 590, 0] + [512] * 8, [300] * 20 + [0] * 50 + [128] * 10])
def test_many_wide_tiles_grouped_rows(lib, dtype, counts):
    import torch
    rng = np.random.default_rng(21)
    N, K = 2600, 136
    G, off = len(counts), np.concatenate([[0], np.cumsum(counts)])
    M = int(off[-1]) + 500
    a, va = operand(lib, rng, M, K, "e4m3")
    b, vb = operand(lib, rng, N, K, "e4m3", G)
    s = 2.0 ** -8
    a = lib.fp8_quantize(torch.from_numpy((va * s).astype(np.float32)).cuda())
    va = values(a)
    out = torch.full((M, N), 7.0, dtype=dt(torch, dtype), device="cuda")
    lib.fp8_matmul(a, b, out=out, offsets=torch.from_numpy(off.astype(np.int32)).cuda())
    torch.cuda.synchronize()
    assert torch.all(out[int(off[-1]):] == 7.0)
    got = host(out)
    for g in range(G):
        lo, hi = off[g], off[g + 1]
        for n in range(0, N, 500):      # a part of the columns at a time
            check_product(got[lo:hi, n:n + 100], va[lo:hi], vb[g][n:n + 100], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_many_wide_tiles_grouped_contraction(lib, dtype):
    # contractions that start and end anywhere in the 16-block parts of the scales
    import torch
    rng = np.random.default_rng(22)
    blocks = ([0, 1, 3, 0, 2, 5, 1, 4, 17, 1, 15, 16, 0, 33] * 5)[:64]
    off = 128 * np.concatenate([[0], np.cumsum(blocks)])
    M, N, K = 512, 480, int(off[-1]) + 1
    a, va = operand(lib, rng, M, K, "e5m2")
    b, vb = operand(lib, rng, N, K, "e4m3")
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    out = torch.empty(len(blocks), M, N, dtype=dt(torch, dtype), device="cuda")
    assert kinds(lib, lambda: lib.fp8_matmul_grouped_k(a, b, offsets, out=out)) == {"fp8_gemm_256"}
    torch.cuda.synchronize()
    got = host(out)
    for g in range(len(blocks)):
        sl = slice(off[g], off[g + 1])
        check_product(got[g][::7], va[::7, sl], vb[:, sl], dtype)


def test_groups_without_columns_ignore_their_neighbours(lib):
    # an empty group gives zeros even where the columns around it hold NaN, and a group of
    # an odd number of blocks does not take in the next group's
    import torch
    rng = np.random.default_rng(23)
    x = rng.standard_normal((512, 128 * 9)).astype(np.float32)
    x[:, 128 * 3:128 * 6] = np.nan
    a = lib.fp8_quantize(torch.from_numpy(x).cuda(), "e5m2")
    b, vb = operand(lib, rng, 512, 128 * 9, "e4m3")
    off = [0, 3, 3, 6, 6, 9] + [9] * 60
    for part in (slice(0, 512), slice(0, 40)):
        aa = lib.Fp8(a.data[part].contiguous(), a.scale[part].contiguous(), a.cols)
        got = host(lib.fp8_matmul_grouped_k(aa, b, (128 * torch.tensor(off, dtype=torch.int32)).cuda(),
                                            out_dtype=torch.float32))
        va = values(aa)
        for g, (lo, hi) in enumerate(zip(off, off[1:])):
            if lo == 3 and hi == 6:
                assert np.all(np.isnan(got[g]))
            elif lo == hi:
                assert np.all(got[g] == 0)
            else:
                check_product(got[g], va[:, 128 * lo:128 * hi], vb[:, 128 * lo:128 * hi], "f32")


def test_long_contraction_and_far_rows(lib):
    # more blocks than the parts of the scales hold twice, rows whose bytes lie beyond 2^32
    import torch
    rng = np.random.default_rng(24)
    K = 128 * 70 + 5
    a, va = operand(lib, rng, 300, K, "e4m3")
    b, vb = operand(lib, rng, 200, K, "e4m3")
    for dtype in ("f32", "bf16"):
        c = lib.fp8_matmul(a, b, out_dtype=dt(torch, dtype))
        check_product(host(c), va, vb, dtype)
    rows, K = (1 << 32) // 4096 + 300, 4096
    big = lib.fp8_empty(rows, K)
    big.data.view(torch.uint8).zero_()
    big.scale.view(torch.uint8).fill_(127)
    tail, vt = operand(lib, rng, 260, K, "e4m3")
    big.data[-260:] = tail.data
    big.scale[-260:] = tail.scale
    w, vw = operand(lib, rng, 48, K, "e4m3")
    c = lib.fp8_matmul(big, w)
    assert torch.all(c[:-260] == 0)
    check_product(host(c[-260:]), vt, vw, "bf16")
    c = lib.fp8_matmul(w, big)
    check_product(host(c[:, -260:]), vw, vt, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(3, 40), (40, 40), (512, 512)])
def test_last_groups_without_columns(lib, M, N, dtype):
    # they begin behind the operand's last block: nothing there is read, also where the
    # last block is not the last of four
    import torch
    rng = np.random.default_rng([M, 25])
    a, va = operand(lib, rng, M, 128 * 5, "e4m3")
    b, vb = operand(lib, rng, N, 128 * 5, "e4m3")
    off = [0, 5] + [5] * 62
    out = torch.full((len(off) - 1, M, N), 7.0, dtype=dt(torch, dtype), device="cuda")
    lib.fp8_matmul_grouped_k(a, b, (128 * torch.tensor(off, dtype=torch.int32)).cuda(), out=out)
    check_product(host(out[0]), va, vb, dtype)
    assert torch.all(out[1:] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(129, 130), (257, 300)])
def test_last_tile_fetches_nothing_more(lib, M, N, dtype):
    # the last tiles' contraction begins in the middle of the operands (beyond the first 16
    # blocks too); behind them a workgroup fetches nothing
    import torch
    rng = np.random.default_rng([M, 26])
    off = [0, 1, 19, 20, 37]
    a, va = operand(lib, rng, M, 128 * 37, "e4m3")
    b, vb = operand(lib, rng, N, 128 * 37, "e5m2")
    got = host(lib.fp8_matmul_grouped_k(a, b, (128 * torch.tensor(off, dtype=torch.int32)).cuda(),
                                        out_dtype=dt(torch, dtype)))
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        check_product(got[g], va[:, 128 * lo:128 * hi], vb[:, 128 * lo:128 * hi], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("M,N", [(512, 512), (300, 260)])
def test_many_groups_of_very_different_length(lib, M, N, dtype):
    # several rounds of tiles and more than 64 groups: they are taken in another order
    import torch
    rng = np.random.default_rng([M, 27])
    blocks = rng.integers(0, 5, 150)
    blocks[rng.random(150) < 0.1] = 11
    blocks[64:80] = 0
    off = np.concatenate([[0], np.cumsum(blocks)])
    a, va = operand(lib, rng, M, 128 * int(off[-1]), "e5m2")
    b, vb = operand(lib, rng, N, 128 * int(off[-1]), "e4m3")
    out = torch.full((150, M, N), 7.0, dtype=dt(torch, dtype), device="cuda")
    lib.fp8_matmul_grouped_k(a, b, (128 * torch.from_numpy(off.astype(np.int32))).cuda(), out=out)
    out = out[:, ::37].cpu()
    for g, (lo, hi) in enumerate(zip(off, off[1:])):
        sl = slice(128 * lo, 128 * hi)
        check_product(host(out[g]), va[::37, sl], vb[:, sl], dtype)
