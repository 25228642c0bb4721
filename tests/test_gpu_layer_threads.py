"""GPU: the expert and 8-bit operators from two threads at once, on one stream and on two,
next to steps with the workspace that the binding keeps: everybody gets what they get alone."""
import threading

import pytest

from test_gpu_moe_layer import flat, layer, layer_inputs

pytestmark = pytest.mark.gpu


def run_all(jobs):
    """Each job in a thread of its own, started together."""
    start, errors = threading.Barrier(len(jobs)), []

    def run(job):
        try:
            start.wait()
            job()
        except Exception as e:          # surfaced in the main thread
            errors.append(e)
    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("own_streams", [False, True])
def test_two_layers_and_steps(lib, own_streams):
    import torch
    K, H, N = 4, 256, 160
    setups = []
    for T, E, seed in ((1600, 16, 3), (9000, 40, 4)):
        x, logits, dy, params, stride = layer_inputs(T, E, H, N, seed)
        setups.append((x, logits, dy, params, stride, E, K, N, torch.zeros(E * stride, dtype=torch.bfloat16, device="cuda")))
    shapes = [(0, 384, 512), (384 * 512, 96, 700)]
    n = 384 * 512 + 96 * 700
    g = (torch.randn(n, device="cuda") * 1e-2).bfloat16()
    p0 = torch.randn(n, device="cuda")
    hyper = lib.hyper(ns_method="standard", ns_dtype="bf16", grad_dtype="bf16", lr=0.02)
    rounds = 8

    def alone(k):
        return [t.clone() for t in flat(layer(lib, *setups[k]), setups[k][8])]

    def steps(p, m):
        for _ in range(4 * rounds):
            lib.step(p, g, m, shapes, hyper)
    want = [alone(0), alone(1)]
    p, m = p0.clone(), torch.zeros_like(p0)
    steps(p, m)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() if own_streams else torch.cuda.current_stream() for _ in range(3)]
    got = [None, None]
    p2, m2 = p0.clone(), torch.zeros_like(p0)
    torch.cuda.synchronize()

    def layers(k):
        with torch.cuda.stream(streams[k]):
            got[k] = [alone(k) for _ in range(rounds)]

    def stepping():
        with torch.cuda.stream(streams[2]):
            steps(p2, m2)
    run_all([lambda: layers(0), lambda: layers(1), stepping])
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            for a, b in zip(r, want[k]):
                same = torch.equal(torch.nan_to_num(a), torch.nan_to_num(b)) if a.is_floating_point() else torch.equal(a, b)
                assert same, k
    assert torch.equal(p, p2) and torch.equal(m, m2)
