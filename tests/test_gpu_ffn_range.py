"""Gated FFN gradients over the whole range of the stored types: inputs of
every size against the fp64 oracle.

The bounds are those of an fp32 evaluation whose operands of a second product
are rounded to the stored type, all of them relative to the sizes of the
terms (u, e as in test_gpu_layers.py):
  * g, u: a sum of D terms in any order;
  * act(g): the logistic, error or tanh function is within 2^-20 of itself
    (hardware exponential and reciprocal), so g times it within 2^-18·|g|;
    act'(g) is a sum of terms of order 1, each with such an error and times at
    most 17 (from there on the function is exactly 0 or 1): within 2^-16;
  * an error eg of g moves act by at most 1.13·eg, and act' by at most 0.8·eg
    and never by more than 1.3; not at all (below 30·e^-30) where |g| is above
    eg + 30;
  * the factors kept for the backward pass are within 2^-10 of themselves.
"""
import numpy as np
import pytest
import torch

import oracle.layers as ol
from test_gpu_layers import DTYPES, E, NAMES, TINY, UNIT, check, f64, ffn_inputs

pytestmark = pytest.mark.gpu


def relative_errors(f, x, wg, wu, wd, dy, dtype):
    u = UNIT[dtype]
    D, F, T = x.shape[1], wd.shape[1], x.shape[0]
    ab = np.abs
    eg, eu = 1.01 * D * E * (ab(x) @ ab(wg).T), 1.01 * D * E * (ab(x) @ ab(wu).T)
    eb = 1.13 * eg + 2.0 ** -18 * ab(f["g"])
    ed = np.where(ab(f["g"]) > eg + 30, 0.0, np.minimum(0.8 * eg, 1.3)) + 2.0 ** -16
    ea = ab(f["u"]) * ed + 1.2 * eu
    eh = 1.01 * (ab(f["u"]) * eb + ab(f["b"]) * eu + eb * eu + u * ab(f["h"])) + TINY
    ea, eb = ea + 1.01 * 2.0 ** -10 * ab(f["a"]) + TINY, eb + 1.01 * 2.0 ** -10 * ab(f["b"]) + TINY
    edh = 1.01 * D * E * (ab(dy) @ ab(wd))
    edg = 1.01 * (ab(f["dh"]) * ea + ab(f["a"]) * edh + ea * edh + u * ab(f["dg"])) + TINY
    edu = 1.01 * (ab(f["dh"]) * eb + ab(f["b"]) * edh + eb * edh + u * ab(f["du"])) + TINY
    k = 1.01 * (2 * max(D, F, T) + 8) * E
    b = {"y": (eh + k * ab(f["h"])) @ ab(wd).T + u * ab(f["y"]),
         "dx": (edg + k * ab(f["dg"])) @ ab(wg) + (edu + k * ab(f["du"])) @ ab(wu) + u * ab(f["dx"]),
         "dw_gate": (edg + k * ab(f["dg"])).T @ ab(x) + u * ab(f["dw_gate"]),
         "dw_up": (edu + k * ab(f["du"])).T @ ab(x) + u * ab(f["dw_up"]),
         "dw_down": ab(dy).T @ (eh + k * ab(f["h"])) + u * ab(f["dw_down"])}
    return {n: 1.02 * v + TINY for n, v in b.items()}


def run(lib, ts, act, dtype):
    f = ol.gated_ffn_grad(f64(ts[4]), *(f64(t) for t in ts[:4]), act)
    b = relative_errors(f, *(f64(t) for t in ts), dtype)
    x, wg, wu, wd, dy = (t.cuda() for t in ts)
    y, saved = lib.muon_gated_ffn(x, wg, wu, wd, act, save=True)
    check(y, f["y"], b["y"], "y")
    for n, g in zip(NAMES, lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved)):
        check(g, f[n], b[n], n)


# few tokens; both tile sizes without and with k splits, widths on and off
# whole 16-byte chunks
SIZES = [(5, 24, 40), (70, 96, 136), (300, 72, 201), (33, 264, 1000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ol.ACTIVATIONS)
@pytest.mark.parametrize("exponent", [-40, -32, -20, 20, 34, 40])
@pytest.mark.parametrize("tokens,model,hidden", SIZES)
def test_scaled_inputs(lib, tokens, model, hidden, exponent, act, dtype):
    """Small and large activations: no factor is lost or overflows."""
    x, *rest = ffn_inputs(tokens, model, hidden, dtype)
    run(lib, (x * 2.0 ** exponent, *rest), act, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ol.ACTIVATIONS)
def test_rows_of_different_sizes(lib, act, dtype):
    """Tokens from 2^-34 to 2^34 beside one another: each gets the gradient
    of its own size."""
    x, wg, wu, wd, dy = ffn_inputs(69, 96, 136, dtype)
    rows = torch.arange(-34, 35, dtype=torch.float32).exp2().to(dtype)
    run(lib, (x * rows[:, None], wg, wu, wd, dy), act, dtype)


@pytest.mark.parametrize("act", ol.ACTIVATIONS)
def test_large_tile_scaled(lib, act):
    """The 256-row tiles: x and dy scaled by powers of two.  Where every gate
    is saturated the block is bilinear in x, so the gradients of x·2^20 are
    those of x·2^36 times powers of two, but for the few gates near zero."""
    dtype = torch.bfloat16
    x, wg, wu, wd, dy = (t.cuda() for t in ffn_inputs(4096, 1024, 4096, dtype))
    got = []
    for e in (20, 36):
        y, saved = lib.muon_gated_ffn(x * 2.0 ** e, wg, wu, wd, act, save=True)
        g = lib.muon_gated_ffn_grad(dy, x * 2.0 ** e, wg, wu, wd, saved)
        got.append([y.double() * 2.0 ** (-2 * e)] + [t.double() * 2.0 ** (-e if n == "dx" else -2 * e)
                                                     for n, t in zip(NAMES, g)])
    for n, a, b in zip(("y", *NAMES), *got):
        assert bool(torch.isfinite(b).all()), n
        # both are within 5e-3 (2-norm) of the exact result; gates with |g| below
        # 30 at 2^20 are one in 2^15
        assert float((a - b).norm()) <= 1e-2 * float(a.norm()), n


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_and_infinity_reach_the_gradients(lib, dtype):
    """A factor that is not finite is kept as such: the gradients of its
    token say so, and no other token's."""
    x, wg, wu, wd, dy = (t.cuda() for t in ffn_inputs(70, 96, 136, dtype))
    x[3, 1] = float("nan")
    x[50, 2] = float("inf")
    _, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True)
    dx, *dw = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved)
    good = [i for i in range(70) if i not in (3, 50)]
    assert torch.isfinite(dx[good]).all() and torch.isnan(dx[3]).all() and not torch.isfinite(dx[50]).any()
    assert all(torch.isnan(g).any() for g in dw)
