"""Workspace sizes of the gated FFN for weights of any alignment (no GPU
needed)."""
import ctypes

import pytest
import torch

import muon_newton_schulz_06_amd as mns
from muon_newton_schulz_06_amd import layers

SIZES = [(1, 64, 96), (70, 64, 96), (70, 96, 136), (300, 72, 200), (300, 33, 50), (2048, 3584, 18944)]


def needed(tokens, model, hidden, grad, addresses, lds):
    """What the library asks for, given the weights' addresses and strides."""
    f = layers.MuonFfn(tokens, model, hidden, *addresses, *lds, 1, 0)
    n = ctypes.c_size_t(0)
    assert layers._lib().muon_gated_ffn_workspace_size(ctypes.byref(f), grad, ctypes.byref(n)) == 0
    return n.value


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("tokens,model,hidden", SIZES)
def test_without_weights_it_is_enough_for_any(tokens, model, hidden, grad):
    got = mns.gated_ffn_workspace_size(tokens, model, hidden, torch.bfloat16, grad)
    for off in (0, 2, 8, 16):
        for pad in (0, 1, 8):
            at = [(k << 40) + off for k in (1, 2, 3)]
            assert got >= needed(tokens, model, hidden, grad, at, (model + pad, model + pad, hidden + pad)), (off, pad)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("tokens,model,hidden", SIZES[:4])
def test_with_weights_it_is_what_the_call_needs(tokens, model, hidden, grad):
    for pad in (0, 3, 8):
        bufs = [torch.zeros((r, c + pad), dtype=torch.bfloat16) for r, c in ((hidden, model),) * 2 + ((model, hidden),)]
        ws = [b[:, pad:] for b in bufs]
        got = mns.gated_ffn_workspace_size(tokens, model, hidden, torch.bfloat16, grad, weights=ws)
        assert got == needed(tokens, model, hidden, grad, [w.data_ptr() for w in ws], [w.stride(0) for w in ws])
        assert got <= mns.gated_ffn_workspace_size(tokens, model, hidden, torch.bfloat16, grad)


def test_weights_must_fit_the_sizes():
    w = torch.zeros((96, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mns.gated_ffn_workspace_size(70, 64, 96, weights=(w, w, w))
    with pytest.raises(TypeError):
        mns.gated_ffn_workspace_size(70, 64, 96, weights=(w, w, w.t().contiguous().float()))
