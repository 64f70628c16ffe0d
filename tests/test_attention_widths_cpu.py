"""Heads of no values are refused by name (no GPU needed)."""
import pytest
import torch

import muon_newton_schulz_06_amd as mns
from test_attention_cpu import free  # noqa: F401  (the fixture)


@pytest.mark.parametrize("lead", [(2,), ()])
def test_heads_without_values(free, lead):  # noqa: F811
    q, k, v = torch.zeros(*lead, 3, 8, 0), torch.zeros(*lead, 5, 4, 0), torch.zeros(*lead, 5, 2, 0)
    o, saved = torch.zeros(*lead, 3, 4, 0), torch.zeros(64, dtype=torch.uint8)
    for kw in (dict(), dict(scale=1.0)):
        with pytest.raises(mns.MuonError, match="dim"):
            mns.muon_diff_attention(q, k, v, torch.zeros(4), **kw)
        with pytest.raises(mns.MuonError, match="dim"):
            mns.muon_diff_attention_grad(o, q, k, v, torch.zeros(4), o, saved, **kw)
    assert not free
