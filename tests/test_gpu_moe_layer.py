"""GPU: the operators together, as a training step around the Muon step uses them, and
their duties as library calls (streams, captured graphs, views of the packed buffers).

One mixture-of-experts projection, forward and backward, with 8-bit products:
  route -> order -> quantise routed rows and packed weights -> experts' product ->
  combine; combine gradient -> quantise dy by routed rows -> input gradient, weight
  gradient into the packed gradients -> muon_step on them.
Each call is checked against the float64 oracle on the values the call before it left, so
every check has the tolerance of one operator (see test_gpu_fp8.py, test_gpu_moe.py).
"""
import numpy as np
import pytest

from oracle import fp8 as F
from oracle import moe as R
from test_gpu_fp8 import check_operand, check_product, host, values

pytestmark = pytest.mark.gpu


def layer_inputs(T, E, H, N, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").bfloat16()
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[T // 2] = -float("inf")                  # a padding token
    dy = torch.randn(T, N, generator=g, device="cuda").bfloat16()
    # packed fp32 params of the experts: `up` matrices among others, as a table of entries
    stride = 2 * N * H
    params = torch.randn(E * stride, generator=g, device="cuda") * 0.05
    return x, logits, dy, params, stride


def layer(lib, x, logits, dy, params, stride, E, K, N, grads):
    """One projection forward and backward; everything it computes."""
    import torch
    H = x.shape[1]
    out = {}
    h = lib.route_hyper(score="softmax", top_k=K)
    ids, w = lib.route(logits, h)
    off, counts, rows, pos = lib.expert_order(ids, E, align=128)
    cap = rows.numel()
    weights = params.as_strided((E, N, H), (stride, H, 1))
    wq, wt = lib.fp8_quantize(weights, blocks=True, transposed="both")
    xq, xt = lib.fp8_quantize(x, transposed="both", row_index=rows, row_div=K)
    o = torch.zeros(cap, N, dtype=torch.bfloat16, device=x.device)
    lib.fp8_matmul(xq, wq, out=o, offsets=off)
    y = lib.combine(o, pos, w)
    dw, do = lib.combine_backward(dy, o, pos, w)
    dlogits = lib.route_backward(dw, logits, ids, h)
    # the same rows straight from dy: gathered, weighted, quantised in one pass
    dq, dt = lib.fp8_quantize(dy, "e5m2", transposed="both", row_index=rows, row_div=K, row_weight=w.view(-1))
    dx = torch.zeros(cap, H, dtype=torch.bfloat16, device=x.device)
    lib.fp8_matmul(dq, wt, out=dx, offsets=off)
    lib.fp8_matmul_grouped_k(dt, xt, off, out=grads.as_strided((E, N, H), (stride, H, 1)))
    out.update(ids=ids, w=w, off=off, counts=counts, rows=rows, pos=pos, wq=wq, wt=wt, xq=xq, xt=xt, o=o, y=y, dw=dw,
               do=do, dlogits=dlogits, dq=dq, dt=dt, dx=dx)
    return out


def test_a_layer_and_its_step(lib):
    import torch
    T, E, K, H, N = 300, 8, 2, 200, 136
    x, logits, dy, params, stride = layer_inputs(T, E, H, N, 1)
    grads = torch.full((E * stride,), 7.0, dtype=torch.bfloat16, device="cuda")
    r = layer(lib, x, logits, dy, params, stride, E, K, N, grads)
    torch.cuda.synchronize()

    ids, w = R.route(host(logits), K)
    assert np.array_equal(r["ids"].cpu().numpy(), ids)
    assert np.all(np.abs(host(r["w"]) - w) <= 2.0 ** -24 * w + 1e-12)
    cap = r["rows"].numel()
    off, counts, rows, pos = R.expert_order(ids, E, 128, cap)
    for name, want in (("off", off), ("counts", counts), ("rows", rows), ("pos", pos)):
        assert np.array_equal(r[name].cpu().numpy(), want), name
    wv = host(r["w"])
    xg = F.gather(host(x), rows, K)
    check_operand(r["xq"], *F.quantize(xg, "e4m3"), cap, H)
    check_operand(r["xt"], *F.quantize(xg.T, "e4m3"), H, cap)
    master = host(params).reshape(E, 2, N, H)[:, 0]
    vw = values(r["wq"])
    for e in range(E):
        q, s = F.quantize(master[e], "e4m3", True)
        assert np.array_equal(vw[e], F.dequantize(q, s, H))
        assert np.array_equal(values(r["wt"])[e], vw[e].T)
    vx, o = values(r["xq"]), host(r["o"])
    for e in range(E):
        sl = slice(off[e], off[e + 1])
        check_product(o[sl], vx[sl], vw[e], "bf16")
    assert np.all(o[off[-1]:] == 0)
    want, mag = R.combine(o, pos, wv)
    tol = 2 * K * 2.0 ** -24 * mag
    assert np.all(np.abs(host(r["y"]) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
    dyv = host(dy)
    dw, mag, do, written = R.combine_backward(dyv, o, pos, wv)
    assert np.all(np.abs(host(r["dw"]) - dw) <= (N + 8) * 2.0 ** -24 * mag)
    dl = R.route_backward(host(r["dw"]), host(logits), ids)
    assert np.all(np.abs(host(r["dlogits"]) - dl) <= 2.0 ** -24 * np.abs(dl) + 1e-11 * np.abs(dw).max() * K)
    assert np.all(host(r["dlogits"])[T // 2] == 0)
    dg = F.gather(dyv, rows, K, wv.reshape(-1).astype(np.float32))
    check_operand(r["dq"], *F.quantize(dg, "e5m2"), cap, N)
    check_operand(r["dt"], *F.quantize(dg.T, "e5m2"), N, cap)
    vd, vt, vdt, vxt = values(r["dq"]), values(r["wt"]), values(r["dt"]), values(r["xt"])
    dx, gw = host(r["dx"]), host(grads).reshape(E, 2, N, H)
    for e in range(E):
        sl = slice(off[e], off[e + 1])
        check_product(dx[sl], vd[sl], vt[e], "bf16")
        check_product(gw[e, 0], vdt[:, sl], vxt[:, sl], "bf16")
    assert np.all(gw[:, 1] == 7.0)           # the neighbours in the packed gradients

    # the step takes these gradients as they are; new weights are quantised from its params
    grads.view(E, 2, N, H)[:, 1] = 0.01
    table = [(e * stride + k * N * H, N, H, 0) for e in range(E) for k in (0, 1)]
    mom = torch.zeros_like(params)
    before = params.clone()
    hyper = lib.hyper(ns_method="standard", ns_dtype="bf16", grad_dtype="bf16", lr=0.02)
    lib.step(params, grads, mom, table, hyper)
    torch.cuda.synchronize()
    assert torch.equal(mom, grads.float()) and not torch.equal(params, before)
    wq2, wt2 = lib.fp8_quantize(params.as_strided((E, N, H), (stride, H, 1)), blocks=True, transposed="both", out=r["wq"],
                                out_t=r["wt"])
    assert wq2 is r["wq"] and wt2 is r["wt"]
    q, s = F.quantize(host(params).reshape(E, 2, N, H)[3, 0], "e4m3", True)
    assert np.array_equal(values(wq2)[3], F.dequantize(q, s, H))


def flat(r, grads):
    import torch
    out = [grads]
    for v in r.values():
        out += [v] if isinstance(v, torch.Tensor) else [v.data.view(torch.uint8), v.scale.view(torch.uint8)]
    return out


def same(a, b):
    import torch
    return all(torch.equal(torch.nan_to_num(x) if x.is_floating_point() else x,
                           torch.nan_to_num(y) if y.is_floating_point() else y) for x, y in zip(a, b))


def test_captured_layers_share_nothing(lib):
    # two layers captured on one stream, replayed on two at once, with eager work of the same
    # kind between the replays: every replay gives the eager result for its inputs
    import torch
    E, K, H, N = 16, 4, 256, 160
    T = 1600                                         # enough slots for an order with workspace
    setups, eager = [], []
    for seed in (3, 4):
        x, logits, dy, params, stride = layer_inputs(T, E, H, N, seed)
        grads = torch.zeros(E * stride, dtype=torch.bfloat16, device="cuda")
        setups.append([x, logits, dy, params, stride, E, K, N, grads])
    side = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(side):
        for s in setups:
            layer(lib, *s)                           # warm
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                r = layer(lib, *s)
            graphs.append((g, r))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        want = []
        for k, s in enumerate(setups):
            s[0].copy_(torch.randn(T, H, device="cuda").bfloat16())
            s[1].copy_(torch.randn(T, E, device="cuda"))
            own = s[:8] + [torch.zeros_like(s[8])]
            want.append([t.clone() for t in flat(layer(lib, *own), own[8])])
            s[8].zero_()
        torch.cuda.synchronize()
        for k, (g, r) in enumerate(graphs):
            with torch.cuda.stream(streams[k]):
                g.replay()
        lib.route(setups[0][1], lib.route_hyper(top_k=K))
        torch.cuda.synchronize()
        for k, (g, r) in enumerate(graphs):
            assert same(flat(r, setups[k][8]), want[k]), (turn, k)


def test_streams_and_devices(lib):
    # outputs and workspaces belong to the stream a call runs on; a raw handle takes calls
    # whose outputs are given
    import torch
    ids = torch.randint(0, 32, (4000, 4), device="cuda", dtype=torch.int32)
    want = lib.expert_order(ids, 32)
    x = torch.randn(500, 300, device="cuda")
    a, b = lib.fp8_quantize(x), lib.fp8_quantize(x[:100])
    c = lib.fp8_matmul(a, b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [(lib.expert_order(ids, 32, stream=s), lib.fp8_quantize(x, stream=s), lib.fp8_matmul(a, b, stream=s))
           for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for order, q, m in got:
        assert all(torch.equal(p, r) for p, r in zip(order, want))
        assert torch.equal(q.data.view(torch.uint8), a.data.view(torch.uint8))
        assert torch.equal(m, c)
    raw = streams[0].cuda_stream
    with pytest.raises(ValueError):
        lib.fp8_matmul(a, b, stream=raw)
    out = torch.zeros_like(c)
    torch.cuda.synchronize()
    lib.fp8_matmul(a, b, out=out, stream=raw)
    torch.cuda.synchronize()
    assert torch.equal(out, c)
    with pytest.raises(ValueError):                 # host tensors
        lib.route(torch.zeros(4, 4), lib.route_hyper())
    with pytest.raises(ValueError):
        lib.combine(torch.zeros(4, 8, device="cuda"), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2))


def test_binding_refusals(lib):
    import torch
    x = torch.randn(10, 300, device="cuda")
    a = lib.fp8_quantize(x)
    with pytest.raises(ValueError):
        lib.fp8_quantize(x.t())                      # rows not contiguous
    with pytest.raises(ValueError):
        lib.fp8_quantize(x, transposed="yes")
    with pytest.raises(ValueError):
        lib.fp8_quantize(x, out=lib.fp8_empty(10, 300, "e5m2"))
    with pytest.raises(lib.MuonError):
        lib.fp8_quantize(x, out=lib.fp8_empty(11, 300))
    with pytest.raises(TypeError):
        lib.fp8_quantize(x.double())
    with pytest.raises(TypeError):
        lib.fp8_quantize(x, row_index=torch.zeros(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        lib.fp8_matmul(a, a, accumulate=True)        # nothing to add to
    with pytest.raises(ValueError):
        lib.fp8_matmul(a, a, out=torch.zeros(10, 11, device="cuda"))
    with pytest.raises(lib.MuonError):
        lib.fp8_matmul(a, lib.fp8_quantize(x[:, :200]))
    with pytest.raises(ValueError):
        lib.fp8_matmul(a, a, offsets=torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(lib.MuonError):               # a result that overlaps an operand
        lib.fp8_matmul(a, a, out=a.data.view(torch.bfloat16).view(-1)[:100].view(10, 10))
    with pytest.raises(ValueError):
        lib.expert_order(torch.zeros(4, dtype=torch.int64, device="cuda"), 4)
    with pytest.raises(lib.MuonError):
        lib.expert_order(torch.zeros(4, dtype=torch.int32, device="cuda"), 4, rows=torch.zeros(4, dtype=torch.int32, device="cuda"))
