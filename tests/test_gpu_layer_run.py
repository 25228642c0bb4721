"""GPU: one training step of an attention layer with the library's operators in a row.

Embedding, norm with 8-bit output, joint projection, attention over packed texts, output
projection, norm with the residual; all gradients back to the embedding, some of them straight into
views of joint buffers; clipping into the packed gradients; the Muon and AdamW steps.

Each stage is compared with its definition in 64 bits on the stage's own inputs. A 16-bit result
is off by half a step per value; a sum's operands were rounded where the operator says so, which the
bounds of test_gpu_attention count. Here a relative 2-norm of twice that is enough to see a
wrong operand or a wrong place: 2^-7 for results in bf16, 2^-4 for values in 8 bits.
"""
import numpy as np
import pytest

from oracle import layer as L
from test_gpu_attention import check_backward, check_forward

pytestmark = pytest.mark.gpu

T, VOCAB, C, H, K, D = 300, 500, 256, 4, 2, 64
LENS = [0, 140, 1, 159]
N = (H + 2 * K) * D
SCALE = 16.0


def host(t):
    return t.detach().cpu().double().numpy()


def values(q):
    """What an operand in 8 bits stands for."""
    s = q.scale.float()[:, :q.data.shape[1] // 128].repeat_interleave(128, 1)
    return host(q.data.float() * s)[:, :q.cols]


def near(got, want, bound=2.0 ** -7):
    got = host(got) if hasattr(got, "cpu") else got
    assert np.linalg.norm(got - want) <= bound * np.linalg.norm(want)


class Layer:
    def __init__(self, torch, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def n(*s):
            return torch.randn(*s, generator=g, device="cuda")
        self.table = [(0, N, C, D), (N * C, C, H * D, 0)]   # the joint projection split by head
        self.params = n(N * C + C * H * D) * 0.06
        self.momentum = torch.zeros_like(self.params)
        self.packed = torch.zeros(self.params.numel(), dtype=torch.bfloat16, device="cuda")
        self.w = [self.params[:N * C].view(N, C), self.params[N * C:].view(C, H * D)]
        self.g = [self.packed[:N * C].view(N, C), self.packed[N * C:].view(C, H * D)]
        self.emb, self.n1, self.n2 = 0.06 * n(VOCAB, C), 1 + 0.1 * n(C), 1 + 0.1 * n(C)
        self.adam = [self.emb, self.n1, self.n2]
        self.state = [(torch.zeros_like(p), torch.zeros_like(p)) for p in self.adam]
        self.ids = torch.randint(-1, VOCAB, (T,), generator=g, device="cuda")
        self.off = torch.tensor(np.cumsum([0] + LENS), dtype=torch.int32, device="cuda")
        self.dy = (0.1 * n(T, C)).bfloat16()

    def run(self, lib, torch):
        s = {}
        w8 = [lib.fp8_quantize(w, blocks=True, transposed="both") for w in self.w]
        x0 = lib.embedding(self.ids, self.emb, scale=SCALE, out_dtype=torch.bfloat16)
        n1 = lib.rms_norm(x0, self.n1, fp8="both")
        qkv = lib.fp8_matmul(n1.fp8, w8[0][0])
        heads = qkv.view(T, H + 2 * K, D)
        q, k, v = heads[:, :H], heads[:, H:H + K], heads[:, H + K:]
        o, lse = lib.attention(q, k, v, offsets=self.off)
        o8, o8t = lib.fp8_quantize(o.view(T, H * D), transposed="both")
        a = lib.fp8_matmul(o8, w8[1][0])
        n2 = lib.rms_norm(a, self.n2, residual=x0)
        # backward
        ds, dn2 = lib.rms_norm_backward(self.dy, n2.sum, self.n2, n2.rstd)
        d8, d8t = lib.fp8_quantize(ds, "e5m2", transposed="both")
        do = lib.fp8_matmul(d8, w8[1][1])
        dwo = lib.fp8_matmul(d8t, o8t, out_dtype=torch.float32)
        dqkv = torch.empty_like(qkv)
        dh = dqkv.view(T, H + 2 * K, D)
        lib.attention_backward(do.view(T, H, D), q, k, v, o, lse, offsets=self.off, dq=dh[:, :H], dk=dh[:, H:H + K],
                               dv=dh[:, H + K:])
        e8, e8t = lib.fp8_quantize(dqkv, "e5m2", transposed="both")
        dn = lib.fp8_matmul(e8, w8[0][1])
        x8t = lib.fp8_quantize(n1.y, transposed="only")
        dwqkv = lib.fp8_matmul(e8t, x8t, out_dtype=torch.float32)
        dx0, dn1 = lib.rms_norm_backward(dn, x0, self.n1, n1.rstd, dsum=ds)
        demb = lib.embedding_backward(dx0, self.ids, VOCAB, scale=SCALE)
        small = [torch.empty_like(t) for t in (demb, dn1, dn2)]
        norm = lib.clip_gradients([dwqkv, dwo, demb, dn1, dn2], 1.0, out=self.g + small)
        s.update(locals())
        return s

    def step(self, lib, s):
        h = lib.hyper(ns_method="standard", ns_dtype="bf16", grad_dtype="bf16", lr=0.02, weight_decay=0.1)
        lib.step(self.params, self.packed, self.momentum, self.table, h)
        for p, g, (m, v) in zip(self.adam, s["small"], self.state):
            lib.adamw(p.view(-1), g.view(-1), m.view(-1), v.view(-1))


def test_stages_and_step(lib):
    import torch
    layer = Layer(torch)
    s = layer.run(lib, torch)
    hoff = np.cumsum([0] + LENS)
    near(s["x0"], L.embedding(host(layer.ids), host(layer.emb), SCALE))
    near(s["n1"].y, L.rms_norm(host(s["x0"]), host(layer.n1))[0])
    near(values(s["n1"].fp8), host(s["n1"].y), 2.0 ** -4)
    w = [values(q[0]) for q in s["w8"]]
    near(s["qkv"], values(s["n1"].fp8) @ w[0].T)
    check_forward(s["q"], s["k"], s["v"], s["o"], s["lse"], "bf16", offsets=hoff)
    near(s["a"], values(s["o8"]) @ w[1].T)
    near(s["n2"].sum, host(s["a"]) + host(s["x0"]))
    near(s["n2"].y, L.rms_norm(host(s["n2"].sum), host(layer.n2))[0])
    ds, dn2 = L.rms_norm_backward(host(layer.dy), host(s["n2"].sum), host(layer.n2), host(s["n2"].rstd))
    near(s["ds"], ds)
    near(s["dn2"], dn2)
    near(s["do"], values(s["d8"]) @ w[1])
    near(s["dwo"], values(s["d8t"]) @ values(s["o8t"]).T)
    check_backward(s["do"].view(T, H, D), s["q"], s["k"], s["v"], s["o"],
                   [s["dh"][:, :H], s["dh"][:, H:H + K], s["dh"][:, H + K:]], "bf16", offsets=hoff)
    near(s["dn"], values(s["e8"]) @ w[0])
    near(s["dwqkv"], values(s["e8t"]) @ values(s["x8t"]).T)
    dx0, dn1 = L.rms_norm_backward(host(s["dn"]), host(s["x0"]), host(layer.n1), host(s["n1"].rstd), host(s["ds"]))
    near(s["dx0"], dx0)
    near(s["dn1"], dn1)
    near(s["demb"], L.embedding_backward(host(s["dx0"]), host(layer.ids), VOCAB, SCALE)[0])
    grads = [host(s[n]) for n in ("dwqkv", "dwo", "demb", "dn1", "dn2")]
    norm, clipped = L.clip(grads, 1.0)
    assert norm > 1.0 and abs(s["norm"].item() / norm - 1) <= 2.0 ** -23
    for got, want in zip(layer.g + s["small"], clipped):
        near(got, want)
    before = [layer.params.clone()] + [p.clone() for p in layer.adam]
    layer.step(lib, s)
    for new, old in zip([layer.params] + layer.adam, before):
        assert torch.isfinite(new).all() and not torch.equal(new, old)


def test_step_follows_the_gradient(lib):
    """The whole chain's gradient against differences of its own loss <dy, y>: along the gradient of
    the norms' weights, where no rounding to 8 bits stands between (the last norm's weight)."""
    import torch
    layer = Layer(torch, 3)
    s = layer.run(lib, torch)
    g = s["dn2"].clone()
    dy, y0 = host(layer.dy), host(s["n2"].y)
    h = 2.0 ** -4
    layer.n2 += h * g / g.norm()
    up = host(layer.run(lib, torch)["n2"].y)
    # linear in this weight: only the rounding of y to bf16 stands between
    slope = np.sum(dy * (up - y0)) / h
    bound = np.linalg.norm(dy) * 2.0 ** -8 * (np.abs(up).max() + np.abs(y0).max()) / h
    assert abs(slope - float(g.norm())) <= bound


def test_captured_layer(lib):
    import torch
    layer = Layer(torch, 1)
    names = ("n2", "do", "dwo", "dh", "dwqkv", "dx0", "demb", "norm")

    def parts(s):
        return [s["n2"].y] + [s[n] for n in names[1:]] + list(s["small"])
    want = [t.clone() for t in parts(layer.run(lib, torch))] + [layer.packed.clone()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.run(lib, torch)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = layer.run(lib, torch)
    got = parts(s) + [layer.packed]
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        again = parts(layer.run(lib, torch))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want))
