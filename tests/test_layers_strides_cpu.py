"""Which strides the layer calls take (no GPU needed): CPU tensors, and a
stand-in for the library that reads what it is pointed at."""
import contextlib
import ctypes

import numpy as np
import pytest
import torch

import muon_newton_schulz_06_amd as mns
from muon_newton_schulz_06_amd import layers


class Library:
    """Entry points note the float32 rows their inputs point at."""

    def __init__(self):
        self.seen = []

    @staticmethod
    def rows(p, ld, tokens, dim):
        flat = np.ctypeslib.as_array((ctypes.c_float * ((tokens - 1) * ld + dim)).from_address(p))
        return np.lib.stride_tricks.as_strided(flat, (tokens, dim), (4 * ld, 4)).copy()

    def muon_gated_ffn(self, f, x, ldx, *rest):
        self.seen.append(self.rows(x, ldx, f._obj.tokens, f._obj.model))
        return 0

    def muon_gated_ffn_grad(self, f, x, ldx, dy, ldy, *rest):
        self.seen += [self.rows(p, ld, f._obj.tokens, f._obj.model) for p, ld in ((x, ldx), (dy, ldy))]
        return 0

    def muon_rms_norm(self, x, ldx, r, ldr, w, wt, eps, y, ldy, s, lds, rstd, tokens, dim, dt, stream):
        self.seen += [self.rows(p, ld, tokens, dim) for p, ld in ((x, ldx), (r, ldr))]
        return 0

    def muon_rms_norm_grad(self, dy, ldy, s, lds, w, wt, rstd, ds, ldd, dx, ldx, dw, acc, tokens, dim, *rest):
        self.seen += [self.rows(p, ld, tokens, dim) for p, ld in ((dy, ldy), (s, lds), (ds, ldd))]
        return 0

    def muon_embedding_grad(self, dy, ldy, ids, nb, tokens, vocab, dim, *rest):
        self.seen.append(self.rows(dy, ldy, tokens, dim))
        return 0

    def __getattr__(self, name):  # the sizes of workspaces and of `saved`
        def size(*args):
            args[-1]._obj.value = 512
            return 0
        return size


@pytest.fixture
def fake(monkeypatch):
    L = Library()
    monkeypatch.setattr(layers, "_lib", lambda: L)
    monkeypatch.setattr(layers, "_device", lambda t, name: t.device)
    monkeypatch.setattr(layers, "_on", lambda dev, stream: contextlib.nullcontext())
    monkeypatch.setattr(layers, "_raw_stream", lambda index: 7)
    monkeypatch.setattr(layers, "_workspace",
                        lambda n, dev, user, stream: contextlib.nullcontext((torch.empty(n, dtype=torch.uint8), n)))
    return L


def values(*shape, seed=1):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


LAYOUTS = {
    "rows": lambda s: values(6, 8, seed=s),
    "padded rows": lambda s: values(6, 11, seed=s)[:, 2:10],
    "transposed": lambda s: values(8, 6, seed=s).t(),
    "every second": lambda s: values(6, 16, seed=s)[:, ::2],
    "one row": lambda s: values(8, 6, seed=s).t()[:1],
    "one row for all": lambda s: values(8, seed=s).expand(6, 8),
    "one value for all": lambda s: values(1, seed=s).expand(6, 8),
    "overlapping rows": lambda s: values(40, seed=s).as_strided((6, 8), (5, 1)),
    "3-D": lambda s: values(2, 3, 8, seed=s),
    "3-D, transposed": lambda s: values(3, 2, 8, seed=s).transpose(0, 1),
    "3-D, a view of strided rows": lambda s: values(6, 16, seed=s)[:, ::2].reshape(6, 8).t().t().unflatten(0, (2, 3)),
    "3-D, every second": lambda s: values(2, 3, 16, seed=s)[..., ::2],
    "3-D, one row for all": lambda s: values(8, seed=s).expand(2, 3, 8),
    "3-D, columns first": lambda s: values(8, 6, seed=s).t().unflatten(0, (2, 3)),
    "one dimension": lambda s: values(16, seed=s)[::2],
}


@pytest.mark.parametrize("layout", LAYOUTS)
def test_inputs_of_any_strides(fake, layout):
    """Every input arrives as the rows it stands for, whatever its strides."""
    x, y, z = (LAYOUTS[layout](s) for s in (1, 2, 3))
    want = [t.reshape(-1, 8).numpy() for t in (x, y, z)]
    w, wd = values(10, 8), values(8, 10)
    mns.muon_gated_ffn(x, w, w, wd)
    mns.muon_gated_ffn_grad(y, x, w, w, wd, torch.zeros(512, dtype=torch.uint8))
    mns.muon_rms_norm(x, torch.ones(8), y)
    mns.muon_rms_norm_grad(x, y, torch.ones(8), torch.ones(x.shape[:-1]), dsum=z)
    mns.muon_embedding_grad(x, torch.zeros(x.shape[:-1], dtype=torch.int64), 5)
    order = [0, 0, 1, 0, 1, 0, 1, 2, 0]
    assert len(fake.seen) == len(order)
    for got, k in zip(fake.seen, order):
        assert np.array_equal(got, want[k])


@pytest.mark.parametrize("layout", ["transposed", "every second", "one row for all", "overlapping rows"])
def test_outputs_and_weights_are_not_copied(fake, layout):
    """A result cannot be written to a copy, and a weight is not copied at
    every call: both must have contiguous rows that do not overlap."""
    bad, x, w, wd = LAYOUTS[layout](1), values(6, 8), values(10, 8), values(8, 10)
    with pytest.raises(ValueError):
        mns.muon_gated_ffn(x, w, w, wd, out=bad)
    with pytest.raises(ValueError):
        mns.muon_rms_norm(x, torch.ones(8), x, out=bad)
    with pytest.raises(ValueError):
        mns.muon_rms_norm(x, torch.ones(8), x, sum_out=bad)
    with pytest.raises(ValueError):
        mns.muon_embedding_grad(x, torch.zeros(6, dtype=torch.int64), 6, out=bad)
    with pytest.raises(ValueError):
        mns.muon_gated_ffn(x, bad, bad, values(8, 6))
    with pytest.raises(ValueError):
        mns.muon_embedding(torch.zeros(2, dtype=torch.int64), bad)
    assert not fake.seen


def test_saved_must_be_whole(fake):
    """`saved` is read as the bytes that follow its address."""
    x, w, wd = values(6, 8), values(10, 8), values(8, 10)
    with pytest.raises(ValueError, match="saved"):
        mns.muon_gated_ffn_grad(x, x, w, w, wd, torch.zeros(1024, dtype=torch.uint8)[::2])
    assert not fake.seen
