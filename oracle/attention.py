"""Plain fp64 forms of rotary positions, dropout and differential attention
(numpy, CPU), and the magnitudes from which the tests derive their tolerances."""
from __future__ import annotations

import numpy as np

# ------------------------------------------------------------------- rotary


def rotary(x, freqs, positions, interleaved=False, scale=1.0, inverse=False):
    """x: (batch, tokens, heads, dim); positions: (batch, tokens) integers."""
    n = len(freqs)
    theta = positions.astype(np.float64)[:, :, None, None] * freqs
    c, s = np.cos(theta), np.sin(theta) * (-1 if inverse else 1)
    y = x.copy()
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    a, b = x[..., one], x[..., two]
    y[..., one], y[..., two] = scale * (a * c - b * s), scale * (a * s + b * c)
    return y


# ------------------------------------------------------------------ dropout


def philox4x32_10(counter, key):
    """Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw: Parallel random
    numbers, as easy as 1, 2, 3; 2011).  counter: (n, 4), key: (2,) 32-bit words;
    (n, 4) words."""
    mask = np.uint64(0xFFFFFFFF)
    c = [np.asarray(counter[:, i], np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & mask,
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & mask]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, axis=1).astype(np.uint32)


def dropout_keep(n, p, seed, offset, start=0):
    """Whether each of n elements from number `start`, a multiple of 4, on is kept."""
    block = np.arange(start // 4, start // 4 + (n + 3) // 4, dtype=np.uint64)
    lo, hi = np.uint64(0xFFFFFFFF), np.uint64(32)
    counter = np.stack([block & lo, block >> hi, np.full_like(block, offset & 0xFFFFFFFF),
                        np.full_like(block, (offset >> 32) & 0xFFFFFFFF)], axis=1)
    words = philox4x32_10(counter, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)).reshape(-1)[:n]
    return words.astype(np.float64) >= np.rint(p * 4294967296.0)


def dropout(x, p, seed, offset, residual=None):
    keep = dropout_keep(x.size, p, seed, offset).reshape(x.shape)
    y = np.where(keep, x / (1.0 - p) if p < 1 else 0.0, 0.0)
    return y if residual is None else residual + y


# --------------------------------------------------- differential attention


def spans(tokens, offsets):
    """[(first, last + 1)] of a packed batch's sequences, with offsets outside
    [0, tokens] cut and decreasing ones raised."""
    at = np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, tokens))
    return [(int(a), int(b)) for a, b in zip(at[:-1], at[1:])]


def softmax(s):
    """Over the last axis; -inf is masked, a row of them gives zeros."""
    top = s.max(axis=-1, keepdims=True, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    e[~np.isfinite(s) & (s < 0)] = 0.0
    n = e.sum(axis=-1, keepdims=True)
    return e / np.where(n > 0, n, 1.0)


def _head(q1, q2, k1, k2, v, lam, scale, causal):
    queries, keys = q1.shape[0], k1.shape[0]
    hidden = np.arange(keys)[None, :] > np.arange(queries)[:, None] + keys - queries
    maps = []
    for q, k in ((q1, k1), (q2, k2)):
        s = scale * (q @ k.T)
        if causal:
            s[hidden] = -np.inf
        maps.append(softmax(s))
    return maps, hidden & bool(causal)


def _problems(q, k, offsets):
    """(batch, query rows, key rows) of the independent softmax problems."""
    if offsets is None:
        return [(b, slice(0, q.shape[1]), slice(0, k.shape[1])) for b in range(q.shape[0])]
    return [(0, slice(a, b), slice(a, b)) for a, b in spans(q.shape[1], offsets) if b > a]


def diff_attention(q, k, v, lam, causal=True, scale=None, offsets=None, unit=0.0, e=2.0 ** -24):
    """(out, bound): arrays of (batch, tokens, heads, values), and the error that
    arithmetic in fp32 (unit roundoff e) with probabilities rounded to `unit`
    and a result rounded to `unit` may make in each element."""
    batch, queries, qh, dim = q.shape
    heads, group = qh // 2, qh // k.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    out, bound = np.zeros((batch, queries, heads, 2 * dim)), np.zeros((batch, queries, heads, 2 * dim))
    for b, rows, cols in _problems(q, k, offsets):
        for h in range(heads):
            g = h // group
            qs, ks, vv = [q[b, rows, 2 * h + m] for m in (0, 1)], [k[b, cols, 2 * g + m] for m in (0, 1)], v[b, cols, g]
            (p1, p2), hidden = _head(*qs, *ks, vv, lam[h], scale, causal)
            out[b, rows, h] = (p1 - lam[h] * p2) @ vv
            for p, w, qq, kk in ((p1, 1.0, qs[0], ks[0]), (p2, abs(lam[h]), qs[1], ks[1])):
                rel = unit + probability_error(qq, kk, scale, hidden, e)
                bound[b, rows, h] += w * rel * (p @ np.abs(vv))
            bound[b, rows, h] += (unit + 2 * e) * np.abs(out[b, rows, h])
    return out, bound


def probability_error(q, k, scale, hidden, e):
    """Relative error per row of normalised probabilities in fp32: a score's sum
    of dim products, its scaling and subtraction (of values up to the largest
    score's magnitude, twice: the row's maximum or log-sum has it too), the
    exponential, the sums over the keys, in numerator and denominator."""
    mag = scale * (np.abs(q) @ np.abs(k).T)
    mag[hidden] = 0.0
    size = mag.max(axis=-1, keepdims=True, initial=0.0)
    return 2 * e * (2 * (q.shape[1] + 8) * size + 2 * k.shape[0] + 64)


def diff_attention_grad(dout, q, k, v, lam, causal=True, scale=None, offsets=None, unit=0.0, e=2.0 ** -24):
    """{"dq", "dk", "dv", "dlam"} and their bounds, for arithmetic in fp32 with
    the difference of the maps, dS and the stored results rounded to `unit`; in
    "dlam²" the sum of the squares of dlam's terms, one per row."""
    batch, queries, qh, dim = q.shape
    heads, group = qh // 2, qh // k.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    got = {"dq": np.zeros(q.shape), "dk": np.zeros(k.shape), "dv": np.zeros(v.shape), "dlam": np.zeros(heads)}
    err = {n: np.zeros(a.shape) for n, a in got.items()}
    err["dlam²"] = np.zeros(heads)
    for b, rows, cols in _problems(q, k, offsets):
        for h in range(heads):
            g, la = h // group, lam[h]
            do, vv = dout[b, rows, h], v[b, cols, g]
            maps, hidden = _head(*(q[b, rows, 2 * h + m] for m in (0, 1)), *(k[b, cols, 2 * g + m] for m in (0, 1)), vv,
                                 la, scale, causal)
            nq, nk = do.shape[0], vv.shape[0]
            n = nq * group + nk
            dA = do @ vv.T
            magA = np.abs(do) @ np.abs(vv).T
            rel = [probability_error(q[b, rows, 2 * h + m], k[b, cols, 2 * g + m], scale, hidden, e) for m in (0, 1)]
            # the row sums δ from stored results: each rounded, with its own error
            err_o = [r + unit for r in rel]
            # Σ_d |dO| Σ_j P|v|
            wide = [(np.abs(do) * (maps[m] @ np.abs(vv))).sum(axis=-1, keepdims=True) for m in (0, 1)]
            d2_err = (err_o[1] + unit + 2 * (dim + 4) * e) * wide[1]
            d1_err = (err_o[0] + unit + 2 * (dim + 4) * e) * wide[0] + 2 * abs(la) * d2_err
            A = maps[0] - la * maps[1]
            got["dv"][b, cols, g] += A.T @ do
            err["dv"][b, cols, g] += (unit * np.abs(A) + rel[0] * maps[0] + abs(la) * rel[1] * maps[1]
                                      + 2 * n * e * (maps[0] + abs(la) * maps[1])).T @ np.abs(do)
            for m, (p, d_err, w) in enumerate(zip(maps, (d1_err, d2_err), (1.0, -la))):
                delta = (p * dA).sum(axis=-1, keepdims=True)
                dS = w * p * (dA - delta)
                big = np.abs(w) * p * (magA + wide[m])
                e_dS = unit * np.abs(dS) + np.abs(w) * p * d_err + (rel[m] + 4 * (dim + 4) * e) * big
                # a row that sees one key: exactly no gradient.  (Not one whose other keys'
                # probabilities vanish, in fp64 below e^-745: P = 1 too, but dA and δ are
                # two roundings of one sum, e_dS apart.)
                lone = (~hidden).sum(axis=-1, keepdims=True) <= 1
                e_dS = np.where(lone, 0.0, e_dS)
                qq, kk = q[b, rows, 2 * h + m], k[b, cols, 2 * g + m]
                got["dq"][b, rows, 2 * h + m] = scale * dS @ kk
                err["dq"][b, rows, 2 * h + m] = scale * (e_dS + 2 * n * e * np.abs(dS)) @ np.abs(kk)
                got["dk"][b, cols, 2 * g + m] += scale * dS.T @ qq
                err["dk"][b, cols, 2 * g + m] += scale * (e_dS + 2 * n * e * np.abs(dS)).T @ np.abs(qq)
                if m == 1:
                    got["dlam"][h] -= delta.sum()
                    err["dlam²"][h] += ((p * np.abs(dA)).sum(axis=-1) ** 2).sum()
                    terms = (p * magA).sum(axis=-1, keepdims=True) + wide[1]
                    err["dlam"][h] += ((2 * rel[1] + (4 * dim + 2 * nk + 2 * batch * queries + 64) * e) * terms).sum()
    for name in ("dq", "dk", "dv"):
        err[name] += (unit + 2 * e) * np.abs(got[name])
    return got, err


# What the roundings of bf16 tensors leave in the mean: a rounding is off by a
# uniform part of half a step, in the mean square by at most u²/3 of the value
# (where it is a power of two, less elsewhere), and independent of the others, so
# mean squares add.  The results' own rounding is not estimated: it is known.


def bf16(x):
    """Rounded to nearest, ties to even, by the upper 16 bits of fp32."""
    b = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    b = (b + 0x7FFF + ((b >> 16) & 1)) >> 16 << 16
    return b.astype(np.uint32).view(np.float32).astype(np.float64)


def diff_attention_spread(dout, q, k, v, lam, causal=True, scale=None, offsets=None, few=False, u=2.0 ** -8):
    """Mean squares of the errors of "out", "dq", "dk", "dv" before their own
    rounding, element by element, where
      – the forward pass takes its probabilities as operands of u, or u² with
        `few`, and divides by the sum of what it takes: O = Σ P(1 + ε)v / Σ P(1 + ε)
        is off by Σ P·ε·(v − O);
      – δ = dout·O is formed from that O, kept in whole multiples of 2^-15 of its
        row's largest value (off by less than one of them): by Σ P·ε·(dA − δ) and
        Σ_d dout·(2^-15 max|O|);
      – the backward pass rounds A = P_1 − λ·P_2 and dS = P·(dA − δ) to u."""
    batch, queries, qh, dim = q.shape
    heads, group = qh // 2, qh // k.shape[2]
    scale = dim ** -0.5 if scale is None else scale
    got = {"out": np.zeros((batch, queries, heads, 2 * dim)), "dq": np.zeros(q.shape), "dk": np.zeros(k.shape),
           "dv": np.zeros(v.shape)}
    w, wp = u * u / 3, (u * u if few else u) ** 2 / 3
    for b, rows, cols in _problems(q, k, offsets):
        for h in range(heads):
            g, la, do, vv = h // group, lam[h], dout[b, rows, h], v[b, cols, h // group]
            qs, ks = [q[b, rows, 2 * h + m] for m in (0, 1)], [k[b, cols, 2 * g + m] for m in (0, 1)]
            maps, hidden = _head(*qs, *ks, vv, la, scale, causal)
            dA, lone = do @ vv.T, (~hidden).sum(axis=-1, keepdims=True) <= 1
            got["dv"][b, cols, g] += w * ((maps[0] - la * maps[1]) ** 2).T @ do ** 2
            for m, (p, c) in enumerate(zip(maps, (1.0, la * la))):
                o, delta, p2 = p @ vv, (p * dA).sum(axis=-1, keepdims=True), p * p
                got["out"][b, rows, h] += c * wp * (p2 @ vv ** 2 - 2 * o * (p2 @ vv) + o ** 2 * p2.sum(axis=-1, keepdims=True))
                step = 2.0 ** -15 * np.abs(o).max(axis=-1, keepdims=True, initial=0.0)
                row = wp * (p2 * (dA - delta) ** 2).sum(axis=-1, keepdims=True) + step ** 2 * (do ** 2).sum(axis=-1, keepdims=True)
                own = np.where(lone, 0.0, c * scale * scale * w * p2 * (dA - delta) ** 2)
                row = np.where(lone, 0.0, c * scale * scale * row)
                got["dq"][b, rows, 2 * h + m] = own @ ks[m] ** 2 + row * (p @ ks[m]) ** 2
                got["dk"][b, cols, 2 * g + m] += (own + row * p2).T @ qs[m] ** 2
    return got


def spread_tolerance(ref, square):
    """2-norm of the error of a bf16 result: its own rounding and the mean squares
    of what came before.  A tenth more for the sample (thousands of errors of either
    size), 2^-17 for the fp32 arithmetic."""
    own = ((bf16(ref) - ref) ** 2).sum()
    return 1.1 * np.sqrt(own + square.sum()) + 2.0 ** -17 * np.sqrt((ref ** 2).sum())
