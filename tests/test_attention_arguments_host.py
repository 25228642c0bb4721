"""Heads without columns are refused as other unsupported head dimensions are, whatever the scale."""
import pytest

import newton_schulz_step_amd as nss
from newton_schulz_step_amd import _binding as B


@pytest.mark.parametrize("scale", [None, 0.5])
@pytest.mark.parametrize("dim", [0, 4])
def test_dimension(dim, scale):
    torch = pytest.importorskip("torch")
    q = torch.empty(3, 2, dim, dtype=torch.bfloat16)
    rows = B._attention_rows(q, q, q, None, True, 0, scale)
    with pytest.raises(nss.MuonError, match="dim must be"):
        B._attention_workspace(rows, 0)
