"""GPU: norm, embedding, clipping and attention on raw stream handles with every result and
workspace given, two captured graphs replayed in turn, and the C calls without optional results.
"""
import ctypes

import pytest

from newton_schulz_step_amd import _binding as B

pytestmark = pytest.mark.gpu


def inputs(seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*s):
        return torch.randn(*s, generator=g, device="cuda")
    lens = [300, 0, 129, 1, 270]
    off = torch.zeros(len(lens) + 66, dtype=torch.int32, device="cuda")   # more than 64 sequences: a list in the workspace
    off[1:len(lens) + 1] = torch.cumsum(torch.tensor(lens), 0)
    off[len(lens) + 1:] = sum(lens)
    return dict(x=n(200, 1000).bfloat16(), r=n(200, 1000).bfloat16(), w=n(1000), dy=n(200, 1000).bfloat16(),
                ids=torch.randint(-1, 900, (6000,), generator=g, device="cuda"), table=n(900, 70), de=n(6000, 70).bfloat16(),
                grads=[n(9000), n(77), n(40000)], q=n(700, 8, 64).bfloat16(), k=n(700, 2, 64).bfloat16(),
                v=n(700, 2, 64).bfloat16(), do=n(700, 8, 64).bfloat16(), off=off)


def run(lib, d):
    import torch
    n = lib.rms_norm(d["x"], d["w"], residual=d["r"])
    dx, dw = lib.rms_norm_backward(d["dy"], n.sum, d["w"], n.rstd)
    y = lib.embedding(d["ids"], d["table"])
    dt = lib.embedding_backward(d["de"], d["ids"], 900)
    outs = [torch.empty_like(t) for t in d["grads"]]
    norm = lib.clip_gradients(d["grads"], 3.0, out=outs)
    o, lse = lib.attention(d["q"], d["k"], d["v"], offsets=d["off"])
    return [n.y, n.sum, n.rstd, dx, dw, y, dt, norm, *outs, o, lse,
            *lib.attention_backward(d["do"], d["q"], d["k"], d["v"], o, lse, offsets=d["off"])]


def test_raw_stream(lib):
    import torch
    d = inputs(1)
    want = run(lib, d)
    got = [torch.full_like(t, 7) for t in want]
    y, total, rstd, dx, dw, e, dt, norm, o1, o2, o3, o, lse, dq, dk, dv = got
    sumsq = torch.zeros((), dtype=torch.float64, device="cuda")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    s = side.cuda_stream
    lib.rms_norm(d["x"], d["w"], residual=d["r"], out=y, out_sum=total, rstd=rstd, stream=s)
    lib.rms_norm_backward(d["dy"], total, d["w"], rstd, dx=dx, dweight=dw, ws=ws, stream=s)
    lib.embedding(d["ids"], d["table"], out=e, stream=s)
    lib.embedding_backward(d["de"], d["ids"], 900, out=dt, ws=ws, stream=s)
    lib.grad_sumsq(d["grads"], out=sumsq, ws=ws, stream=s)
    lib.clip_gradients(d["grads"], 3.0, sumsq=sumsq, out=[o1, o2, o3], norm=norm, stream=s)
    lib.attention(d["q"], d["k"], d["v"], offsets=d["off"], out=o, lse=lse, ws=ws, stream=s)
    lib.attention_backward(d["do"], d["q"], d["k"], d["v"], o, lse, offsets=d["off"], dq=dq, dk=dk, dv=dv, ws=ws, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # what would have to be allocated is refused
    for call in (lambda: lib.rms_norm(d["x"], stream=s), lambda: lib.embedding(d["ids"], d["table"], stream=s),
                 lambda: lib.rms_norm_backward(d["dy"], total, d["w"], rstd, dx=dx, dweight=dw, stream=s),
                 lambda: lib.embedding_backward(d["de"], d["ids"], 900, out=dt, stream=s),
                 lambda: lib.clip_gradients(d["grads"], 3.0, norm=norm, stream=s),
                 lambda: lib.attention(d["q"], d["k"], d["v"], offsets=d["off"], out=o, lse=lse, stream=s),
                 lambda: lib.attention_backward(d["do"], d["q"], d["k"], d["v"], o, lse, dq=dq, dk=dk, dv=dv, stream=s)):
        with pytest.raises(ValueError, match="raw stream"):
            call()


def test_two_graphs_in_turn(lib):
    import torch
    data = [inputs(2), inputs(3)]
    want = [[t.clone() for t in run(lib, d)] for d in data]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(lib, data[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs, got = [], []
    for d in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(run(lib, d))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in data]
    for turn in range(4):
        for t in got[0] + got[1]:
            t.zero_()
        torch.cuda.synchronize()
        for i in ((0, 1), (1, 0))[turn % 2]:
            with torch.cuda.stream(streams[i] if turn > 1 else torch.cuda.current_stream()):
                graphs[i].replay()   # at once from the third turn on
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
        assert all(torch.equal(a, b) for a, b in zip(run(lib, data[turn % 2]), want[turn % 2]))


def test_without_optional_results(lib):
    import torch
    d, c = inputs(4), B.load()
    want = run(lib, d)
    s = torch.cuda.current_stream().cuda_stream
    o = torch.empty_like(d["q"])
    a = B._attention_rows(d["q"], d["k"], d["v"], d["off"], True, 0, None)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    heads = [ctypes.byref(B._heads(t, "t")) for t in (d["q"], d["k"], d["v"], o)]
    assert c.muon_attention(ctypes.byref(a), *heads, None, ws.data_ptr(), ws.numel(), s) == 0   # no log-sum-exp
    assert torch.equal(o, want[11])
    rows = B._norm_rows(d["x"], d["w"], d["r"], 1e-6)
    rstd, total = torch.empty_like(want[2]), torch.empty_like(want[1])
    assert c.muon_rms_norm(ctypes.byref(rows), None, 0, None, 0, None, rstd.data_ptr(), s) == 0
    assert c.muon_rms_norm(ctypes.byref(rows), total.data_ptr(), 1000, None, 0, None, None, s) == 0
    assert torch.equal(rstd, want[2]) and torch.equal(total, want[1])
    rows = B._norm_rows(want[1], d["w"], None, 0.0)
    dx, dw = torch.empty_like(want[3]), torch.empty_like(want[4])
    back = [ctypes.byref(rows), want[2].data_ptr(), d["dy"].data_ptr(), 1000, None, 0]
    assert c.muon_rms_norm_backward(*back, dx.data_ptr(), 1000, None, 0, 0, None, 0, s) == 0
    assert c.muon_rms_norm_backward(*back, None, 0, dw.data_ptr(), 0, 0, ws.data_ptr(), ws.numel(), s) == 0
    assert torch.equal(dx, want[3]) and torch.equal(dw, want[4])
