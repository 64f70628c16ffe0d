"""Plain fp64 forms of the layer operators (numpy, CPU), and the size of the
terms of each sum, from which the tests derive their tolerances."""
from __future__ import annotations

import math

import numpy as np

ACTIVATIONS = ("silu", "gelu", "gelu_tanh")


def embedding(ids, weight, scale):
    out = np.zeros((ids.size, weight.shape[1]))
    for t, i in enumerate(ids.ravel()):
        if 0 <= i < weight.shape[0]:
            out[t] = scale * weight[i]
    return out.reshape(*ids.shape, weight.shape[1])


def embedding_grad(dy, ids, vocab, scale):
    """(gradient, Σ|terms|, number of terms per id)."""
    dy = dy.reshape(ids.size, -1)
    dw, mag, n = np.zeros((vocab, dy.shape[1])), np.zeros((vocab, dy.shape[1])), np.zeros(vocab, np.int64)
    for t, i in enumerate(ids.ravel()):
        if 0 <= i < vocab:
            dw[i] += scale * dy[t]
            mag[i] += abs(scale) * np.abs(dy[t])
            n[i] += 1
    return dw, mag, n


def rms_norm(x, weight, residual, eps):
    s = x if residual is None else x + residual
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=-1) + eps)
    return s * rstd[..., None] * weight, s, rstd


def rms_norm_grad(dy, s, weight, rstd, dsum=None):
    n = s * rstd[..., None]
    wd = weight * dy
    c = np.mean(wd * n, axis=-1, keepdims=True)
    dx = rstd[..., None] * (wd - n * c)
    if dsum is not None:
        dx = dx + dsum
    return dx, (dy * n).reshape(-1, dy.shape[-1]).sum(axis=0)


def _erf(x):
    return np.vectorize(math.erf, otypes=[np.float64])(x)


def activation(g, kind):
    """act(g) and act'(g)."""
    with np.errstate(over="ignore"):
        if kind == "silu":
            s = 1.0 / (1.0 + np.exp(-g))
            return g * s, s * (1.0 + g * (1.0 - s))
        if kind == "gelu":
            c = 0.5 * (1.0 + _erf(g / math.sqrt(2.0)))
            return g * c, c + g * np.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
        k = math.sqrt(2.0 / math.pi)
        t = np.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 0.134145 * g * g)


def gated_ffn(x, w_gate, w_up, w_down, kind):
    """Every tensor of the forward pass, by name."""
    g, u = x @ w_gate.T, x @ w_up.T
    v, d = activation(g, kind)
    h = v * u
    return {"g": g, "u": u, "a": u * d, "b": v, "h": h, "y": h @ w_down.T}


def gated_ffn_grad(dy, x, w_gate, w_up, w_down, kind):
    f = gated_ffn(x, w_gate, w_up, w_down, kind)
    dh = dy @ w_down
    dg, du = dh * f["a"], dh * f["b"]
    return {**f, "dh": dh, "dg": dg, "du": du, "dx": dg @ w_gate + du @ w_up,
            "dw_gate": dg.T @ x, "dw_up": du.T @ x, "dw_down": dy.T @ f["h"]}
