"""GPU: the gradients of a whole layer against differences of its loss in 64 bits.

Embedding, norm, joint projection, attention, output projection, norm with the residual, loss
<dy, y>; the projections are fp32 products here, so that no rounding to 8 bits hides a wrong
gradient. Along each parameter's own gradient the loss has the slope |gradient|. 16 roundings
to bf16 lie on the way (forward: rows, normed rows, q k v, probabilities, attention's output, its
projection, the sum, y; backward: the rows' gradient, that of attention's output, score
gradients, probabilities, those of q k v, the normed rows', the rows', and the stored weights'
one in the bound's favour). Each is off by up to 2^-8 of a value, in the mean of squares a root
of three less, and they are independent of each other: six times the root of 16 of them.
"""
import numpy as np
import pytest

from oracle import layer as L

pytestmark = pytest.mark.gpu

T, VOCAB, C, H, K, D = 180, 60, 96, 4, 2, 32
LENS = [70, 0, 1, 109]
SCALE = 4.0
BOUND = 6 * np.sqrt(16) * 2.0 ** -8 / np.sqrt(3)


def host(t):
    return t.detach().cpu().double().numpy()


def loss(p, ids, off, dy):
    x0 = L.embedding(ids, p["emb"], SCALE)
    n1 = L.rms_norm(x0, p["w1"])[0]
    h = (n1 @ p["wqkv"].T).reshape(T, H + 2 * K, D)
    o = L.attention(h[:, :H], h[:, H:H + K], h[:, H + K:], offsets=off)[0]
    y = L.rms_norm(o.reshape(T, H * D) @ p["wo"].T + x0, p["w2"])[0]
    return np.sum(dy * y)


def gradients(lib, torch, p, ids, off, dy):
    b16 = torch.bfloat16
    x0 = lib.embedding(ids, p["emb"], scale=SCALE, out_dtype=b16)
    n1 = lib.rms_norm(x0, p["w1"])
    h = (n1.y.float() @ p["wqkv"].t()).to(b16).view(T, H + 2 * K, D)
    q, k, v = h[:, :H], h[:, H:H + K], h[:, H + K:]
    o, lse = lib.attention(q, k, v, offsets=off)
    n2 = lib.rms_norm((o.view(T, H * D).float() @ p["wo"].t()).to(b16), p["w2"], residual=x0)
    ds, dw2 = lib.rms_norm_backward(dy, n2.sum, p["w2"], n2.rstd)
    do = (ds.float() @ p["wo"]).to(b16)
    dwo = ds.float().t() @ o.view(T, H * D).float()
    dh = torch.empty_like(h)
    lib.attention_backward(do.view(T, H, D), q, k, v, o, lse, offsets=off, dq=dh[:, :H], dk=dh[:, H:H + K], dv=dh[:, H + K:])
    flat = dh.view(T, -1).float()
    dx0, dw1 = lib.rms_norm_backward((flat @ p["wqkv"]).to(b16), x0, p["w1"], n1.rstd, dsum=ds)
    return {"w2": dw2, "wo": dwo, "wqkv": flat.t() @ n1.y.float(), "w1": dw1,
            "emb": lib.embedding_backward(dx0, ids, VOCAB, scale=SCALE)}


def test_slopes_along_the_gradients(lib):
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)

    def n(*s):
        return torch.randn(*s, generator=g, device="cuda")
    p = {"emb": 0.25 * n(VOCAB, C), "w1": 1 + 0.1 * n(C), "w2": 1 + 0.1 * n(C), "wqkv": n((H + 2 * K) * D, C) * C ** -0.5,
         "wo": n(C, H * D) * (H * D) ** -0.5}
    ids = torch.randint(-1, VOCAB, (T,), generator=g, device="cuda")
    off = np.cumsum([0] + LENS)
    dy = (0.1 * n(T, C)).bfloat16()
    got = {k: host(x) for k, x in gradients(lib, torch, p, ids, torch.from_numpy(off.astype(np.int32)).cuda(), dy).items()}
    at = {k: host(x) for k, x in p.items()}
    rows = {"wqkv q": slice(0, H * D), "wqkv k": slice(H * D, (H + K) * D), "wqkv v": slice((H + K) * D, None)}
    for name in ("w2", "wo", "wqkv q", "wqkv k", "wqkv v", "w1", "emb"):
        key = name.split()[0]
        u = np.zeros(at[key].shape)
        u[rows.get(name, slice(None))] = got[key][rows.get(name, slice(None))]
        size = np.linalg.norm(u)
        u *= 1e-5 * np.linalg.norm(at[key]) / size
        step = np.linalg.norm(u)

        def f(sign):
            return loss({**at, key: at[key] + sign * u}, host(ids), off, host(dy))
        slope = (f(1) - f(-1)) / (2 * step)
        assert abs(slope / size - 1) <= BOUND, (name, slope / size)
