"""The tolerances that hold the attention of bf16 tensors to its precision (no
GPU needed): a plain model of the kernels' roundings stays within them, and does
not with any one of the choices that keep it there taken back."""
import numpy as np
import pytest

import oracle.attention as oa

# batch, queries, keys, heads, kv heads, dim, the values' common part, offsets
CASES = {
    "random": (1, 300, 300, 4, 2, 64, 0.0, None),
    "wide": (2, 130, 130, 2, 1, 128, 0.0, None),
    "common": (1, 200, 200, 4, 2, 64, 8.0, None),
    "pairs": (1, 400, 400, 3, 1, 40, 0.0, list(range(0, 401, 2))),
    "threes": (1, 300, 300, 2, 2, 64, 4.0, list(range(0, 301, 3))),
    "wide pairs": (1, 200, 200, 4, 2, 96, 8.0, list(range(0, 201, 2))),
    "one token": (4, 1, 700, 6, 2, 64, 0.0, None),
    "few tokens": (8, 3, 150, 4, 4, 128, 2.0, None),
    "few wide": (8, 2, 150, 4, 4, 128, 0.0, None),
    "two keys": (64, 2, 2, 4, 2, 40, 0.0, None),
}


def few(name):
    """Calls of at most 32 rows per key head take the forward pass of few rows."""
    _, queries, _, heads, kv, *_ = CASES[name]
    return queries * heads // kv <= 32


def inputs(name, seed=90):
    """bf16 values (λ: fp32) in fp64."""
    batch, queries, keys, heads, kv, dim, common, offsets = CASES[name]
    r = np.random.RandomState(seed + list(CASES).index(name))
    q, k, v, do = (oa.bf16(r.randn(*s)) for s in ((batch, queries, 2 * heads, dim), (batch, keys, 2 * kv, dim),
                                                 (batch, keys, kv, 2 * dim), (batch, queries, heads, 2 * dim)))
    return do, q, k, oa.bf16(v + common), (0.2 + 0.6 * r.rand(heads)).astype(np.float32).astype(np.float64), offsets


def errors(got, name, ts=None):
    """{result: its error's 2-norm in units of the tolerance}"""
    do, q, k, v, lam, offsets = ts or inputs(name)
    ref, _ = oa.diff_attention(q, k, v, lam, offsets=offsets)
    refs = {"out": ref, **oa.diff_attention_grad(do, q, k, v, lam, offsets=offsets)[0]}
    square = oa.diff_attention_spread(do, q, k, v, lam, offsets=offsets, few=few(name))
    return {n: np.linalg.norm(got[n] - refs[n]) / oa.spread_tolerance(refs[n], s) for n, s in square.items()}


def model(do, q, k, v, lam, offsets, few, keep16=True, rounded_sum=True, split=True):
    """The kernels' roundings in otherwise exact arithmetic.  keep16: P_m·v kept in
    multiples of 2^-15 of a row's largest, else in bf16; rounded_sum: results
    divided by the sum of the rounded probabilities; split: the probabilities of
    few rows as two operands."""
    batch, queries, qh, dim = q.shape
    heads, group, scale = qh // 2, qh // k.shape[2], dim ** -0.5
    got = {"out": np.zeros(do.shape), "dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape)}
    for b, rows, cols in oa._problems(q, k, offsets):
        for h in range(heads):
            g, la, d, vv = h // group, lam[h], do[b, rows, h], v[b, cols, h // group]
            nq, nk = d.shape[0], vv.shape[0]
            hidden = np.arange(nk)[None, :] > np.arange(nq)[:, None] + nk - nq
            dA, o, p, kept = d @ vv.T, [], [], []
            for m in (0, 1):
                s = np.where(hidden, -np.inf, scale * (q[b, rows, 2 * h + m] @ k[b, cols, 2 * g + m].T))
                # the running maximum may lag behind: here by a factor of up to 8
                e = np.exp(s - s.max(axis=-1, keepdims=True) + np.linspace(0.0, 2.0, nq)[:, None])
                taken = oa.bf16(e)
                if few and split:
                    taken = taken + oa.bf16(e - taken)
                total = (taken if rounded_sum else e).sum(axis=-1, keepdims=True)
                p.append(e / e.sum(axis=-1, keepdims=True))
                o.append(taken @ vv / total)
                unit = np.abs(o[m]).max(axis=-1, keepdims=True) / 32767
                kept.append(np.rint(o[m] / unit) * unit if keep16 else oa.bf16(o[m]))
            got["out"][b, rows, h] = o[0] - la * o[1]
            got["dv"][b, cols, g] += oa.bf16(p[0] - la * p[1]).T @ d
            lone = (~hidden).sum(axis=-1, keepdims=True) <= 1
            for m, w in enumerate((1.0, -la)):
                dS = np.where(lone, 0.0, oa.bf16(p[m] * (dA - (d * kept[m]).sum(axis=-1, keepdims=True))))
                got["dq"][b, rows, 2 * h + m] = w * scale * (dS @ k[b, cols, 2 * g + m])
                got["dk"][b, cols, 2 * g + m] += w * scale * (dS.T @ q[b, rows, 2 * h + m])
    return {n: oa.bf16(t) for n, t in got.items()}


@pytest.mark.parametrize("name", CASES)
def test_model_is_within(name):
    ts = inputs(name)
    found = errors(model(*ts, few(name)), name, ts)
    assert max(found.values()) <= 1.0, found
    assert min(found.values()) >= 0.5, found  # (a tolerance far above what is left would hold nothing)


@pytest.mark.parametrize("mistake,names", [
    (dict(keep16=False), ("pairs", "threes", "wide pairs", "two keys", "common")),
    (dict(rounded_sum=False), ("threes", "wide pairs", "common")),
    (dict(split=False), ("one token", "few wide"))])
def test_mistakes_are_not(mistake, names):
    for name in names:
        ts = inputs(name)
        found = errors(model(*ts, few(name), **mistake), name, ts)
        assert max(found.values()) > 1.0, (name, found)
