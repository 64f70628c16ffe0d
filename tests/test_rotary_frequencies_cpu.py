"""Rotary frequencies that no formula gives are refused as such (no GPU needed)."""
import pytest

import muon_newton_schulz_06_amd as mns


@pytest.mark.parametrize("kw", [dict(base=1.0), dict(base=0.5), dict(fast=0.0), dict(slow=0.0), dict(fast=-1.0), dict(slow=-2.0),
                                dict(original_length=0), dict(original_length=-5), dict(slow=64.0)])
def test_yarn_frequencies(kw):
    """The ramp goes from `fast` turns down to `slow`, which needs frequencies that fall."""
    with pytest.raises(ValueError, match="yarn"):
        mns.rotary_frequencies(64, **{**dict(scaling="yarn", factor=8.0, original_length=2048), **kw})
