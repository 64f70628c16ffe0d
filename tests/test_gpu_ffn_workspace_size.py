"""A workspace of the size the binding names serves weights of any alignment."""
import pytest
import torch

from test_gpu_layers import ffn_inputs, strided

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [5, 70, 300])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_workspace_of_that_size(lib, tokens, pad):
    ts = ffn_inputs(tokens, 96, 136, torch.bfloat16)
    x, wg, wu, wd, dy = (strided(t, pad) for t in ts)
    ref, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True)
    grads = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved)
    for weights in (None, (wg, wu, wd)):
        def ws(grad):
            n = lib.gated_ffn_workspace_size(tokens, 96, 136, torch.bfloat16, grad, weights=weights)
            # what lies beyond it must stay as it is
            return torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda"), n
        fw, n = ws(False)
        y, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True, workspace=fw[:n])
        bw, m = ws(True)
        got = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved, workspace=bw[:m])
        assert torch.equal(y, ref) and all(torch.equal(a, b) for a, b in zip(grads, got))
        assert bool((fw[n:] == 7).all()) and bool((bw[m:] == 7).all())
