"""GPU: orders that take a workspace from several threads on one stream, on a raw handle
and in graphs captured on one."""
import threading

import numpy as np
import pytest

from oracle import moe as R

pytestmark = pytest.mark.gpu


def test_orders_of_two_threads_on_one_stream(lib):
    import torch
    sizes = [(5000, 7), (40000, 64)]
    host_ids = [np.random.default_rng(n).integers(-1, E, n).astype(np.int32) for n, E in sizes]
    ids = [torch.from_numpy(i).cuda() for i in host_ids]
    want = [R.expert_order(i, E, 16, n + E * 15) for i, (n, E) in zip(host_ids, sizes)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def run(k):
        try:
            got[k] = [lib.expert_order(ids[k], sizes[k][1], align=16) for _ in range(100)]
        except Exception as e:          # surfaced in the main thread
            errors.append(e)
    threads = [threading.Thread(target=run, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for k in range(2):
        for order in got[k]:
            assert all(np.array_equal(t.cpu().numpy(), w) for t, w in zip(order, want[k]))


def outputs(n, E, align):
    import torch
    make = lambda m: torch.full((m,), 77, dtype=torch.int32, device="cuda")   # noqa: E731
    return dict(offsets=make(E + 1), counts=make(E), rows=make(n + E * (align - 1)), pos=make(n))


def test_raw_handles_and_their_graphs_take_given_workspaces(lib):
    import torch
    n, E, align = 6000, 20, 16
    rng = np.random.default_rng(0)
    ids = [torch.from_numpy(rng.integers(-1, E, n).astype(np.int32)).cuda() for _ in range(2)]
    side = torch.cuda.Stream()
    raw = side.cuda_stream
    torch.cuda.synchronize()
    with pytest.raises(ValueError, match="workspace"):
        lib.expert_order(ids[0], E, align=align, stream=raw, **outputs(n, E, align))
    with pytest.raises(lib.MuonError):              # one that is too small
        lib.expert_order(ids[0], E, align=align, stream=raw, ws=torch.empty(8, device="cuda"), **outputs(n, E, align))
    small = lib.expert_order(ids[0][:100], E, align=align, stream=raw, **outputs(100, E, align))   # takes none
    torch.cuda.synchronize()
    need = lib.expert_order_workspace_size(n, E)
    graphs = []
    for k in range(2):
        out, ws = outputs(n, E, align), torch.zeros(need, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            lib.expert_order(ids[k], E, align=align, stream=raw, ws=ws, **out)
        graphs.append((g, out, ws))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(3):
        for k in range(2):
            ids[k].copy_(torch.from_numpy(rng.integers(-1, E, n).astype(np.int32)))
        torch.cuda.synchronize()
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k][0].replay()
        torch.cuda.synchronize()
        for k in range(2):
            want = R.expert_order(ids[k].cpu().numpy(), E, align, n + E * (align - 1))
            for got, w in zip(graphs[k][1].values(), want):
                assert np.array_equal(got.cpu().numpy(), w), (turn, k)
    assert int(small[1].sum()) + int((small[3] < 0).sum()) == 100
