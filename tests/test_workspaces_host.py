"""Workspaces of the expert operators without a GPU: a call that passes data from one
launch to the next through a workspace shares it with no other call."""
import pytest

import newton_schulz_step_amd as nss
from newton_schulz_step_amd import _binding as B


def on_host(raw=False):
    """What a call runs on, on the host: only its memory is looked at."""
    import torch
    on = object.__new__(B._on)
    on.dev, on.raw, on._ctx, on._stream = torch.device("cpu"), raw, None, 1234 if raw else None
    return on


def test_two_calls_have_two_workspaces(monkeypatch):
    def refuse(*a, **k):
        raise AssertionError("the workspace that steps share was asked for")
    monkeypatch.setattr(B, "workspace", refuse)
    on = on_host()
    a, b = on.scratch(4096), on.scratch(4096)
    assert a.numel() >= 4096 and b.numel() >= 4096 and a.data_ptr() != b.data_ptr()
    assert on.scratch(0) is None


def test_a_raw_handle_takes_a_given_workspace():
    import torch
    ws = torch.empty(100, dtype=torch.uint8)
    assert on_host(raw=True).scratch(64, ws) is ws and on_host().scratch(64, ws) is ws
    assert on_host(raw=True).scratch(0) is None
    with pytest.raises(ValueError, match="workspace"):
        on_host(raw=True).scratch(64)


def test_workspace_size():
    assert nss.expert_order_workspace_size(4096, 8) == 0
    assert nss.expert_order_workspace_size(4097, 8) >= 2 * 8 * 4
    with pytest.raises(nss.MuonError):
        nss.expert_order_workspace_size(-1, 8)
