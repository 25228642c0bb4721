"""Integers that do not fit the C ABI's 32 bits are refused, not cut: 2^32 + 1 is not 1."""
import pytest

import newton_schulz_step_amd as nss

WIDE = (1 << 32) + 1


@pytest.mark.parametrize("name", ["score", "top_k", "n_groups", "top_groups", "group_top", "renormalize"])
def test_router_hyperparameters(name):
    for bad in (WIDE, -WIDE, 1 << 31):
        with pytest.raises(ValueError, match=name):
            nss.route_hyper(**{name: bad})
    assert getattr(nss.route_hyper(**{name: True}), name) == 1
    with pytest.raises(TypeError):
        nss.route_hyper(**{name: 1.5})


def test_call_arguments():
    # refused before anything is asked about the tensors' device
    import torch
    ids = torch.zeros(4, dtype=torch.int32)
    for kw in (dict(n_experts=WIDE), dict(n_experts=4, align=WIDE)):
        with pytest.raises(ValueError, match="32-bit"):
            nss.expert_order(ids, **kw)
    with pytest.raises(ValueError, match="32-bit"):
        nss.expert_order_workspace_size(5000, WIDE)
    with pytest.raises(ValueError, match="row_div"):
        nss.fp8_quantize(torch.zeros(4, 4), row_index=ids, row_div=WIDE)
