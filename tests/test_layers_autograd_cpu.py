"""The modules' autograd behaviour with stand-ins for the library's calls (no
GPU needed)."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

from muon_newton_schulz_06_amd import layers


@pytest.fixture
def fake(monkeypatch):
    """y = 2x computed outside autograd, as the kernels do; notes `save`."""
    saves = []

    def ffn(x, *w, save=False, **kw):
        saves.append(save)
        y = torch.from_numpy(x.detach().numpy() * 2)
        return (y, torch.zeros(8, dtype=torch.uint8)) if save else y

    def grad(dy, x, wg, wu, wd, saved, want_dx=True, want_dweights=True, **kw):
        return (torch.from_numpy(dy.numpy() * 2) if want_dx else None,
                *(torch.ones_like(w) if want_dweights else None for w in (wg, wu, wd)))
    monkeypatch.setattr(layers, "muon_gated_ffn", ffn)
    monkeypatch.setattr(layers, "muon_gated_ffn_grad", grad)
    return saves


def frozen(ffn):
    for p in ffn.parameters():
        p.requires_grad_(False)
    return ffn


@pytest.mark.parametrize("mode", [torch.no_grad, torch.enable_grad])
@pytest.mark.parametrize("trains", [False, True])
def test_tangents_are_refused(fake, mode, trains):
    """Forward-mode derivatives are not defined: a dual input raises, in every
    mode, and is never answered with a tangent of zero."""
    ffn = layers.GatedFFN(6, 8) if trains else frozen(layers.GatedFFN(6, 8))
    with mode(), fwad.dual_level():
        x = fwad.make_dual(torch.ones(2, 6), torch.ones(2, 6))
        with pytest.raises(NotImplementedError):
            ffn(x)


def test_nothing_is_saved_without_need(fake):
    """What the backward pass reads is kept only where there is one."""
    x = torch.ones(2, 6)
    ffn = layers.GatedFFN(6, 8)
    with torch.no_grad():
        assert torch.equal(ffn(x), 2 * x)
        ffn(x.clone().requires_grad_())
    with torch.inference_mode():
        ffn(x)
    assert not ffn(x.clone().requires_grad_()).detach().requires_grad
    frozen(ffn)
    y = ffn(x)
    assert not y.requires_grad
    ffn(x.clone().requires_grad_())
    assert fake == [False, False, False, True, False, True]


def test_gradients_flow(fake):
    ffn = layers.GatedFFN(6, 8)
    x = torch.ones(2, 6, requires_grad=True)
    ffn(x).sum().backward()
    assert torch.equal(x.grad, torch.full((2, 6), 2.0)) and all((p.grad == 1).all() for p in ffn.parameters())
    frozen(ffn).zero_grad()
    x.grad = None
    ffn(x).sum().backward()
    assert torch.equal(x.grad, torch.full((2, 6), 2.0)) and all(p.grad is None for p in ffn.parameters())
