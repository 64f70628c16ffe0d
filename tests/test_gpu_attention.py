"""Rotary positions, dropout and differential attention against the fp64
oracle.

Tolerances are element-wise bounds derived from the arithmetic, beside the
oracle's forms for the attention.  u is the unit roundoff of the stored type
(bf16 2^-8, fp32 2^-24), e = 2^-24 that of the fp32 arithmetic.

The bounds let every rounding of a sum point the same way.  For the attention
of random values the whole results are held to what roundings of either sign
leave as well: a bf16 result has been through at most four (its operands', the
row sums', its own), of at most u each and less than that in the mean; fp32 sums
of n terms are off by some √n·e, a probability by some 16·e of its score.
"""
import math

import numpy as np
import pytest
import torch

import oracle.attention as oa

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
UNIT = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}
TINY = 2.0 ** -120  # results this small may be flushed
DTYPES = [torch.bfloat16, torch.float32]


def rand(shape, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def place(t, layout="bthd", pad=0, start=0):
    """The same (batch, tokens, heads, values) on the GPU, dimensions in memory
    in the order of `layout`, `pad` elements behind every head and `start` in
    front of the first.  What lies between holds NaN: reading it shows."""
    order = ["bthd".index(c) for c in layout]
    shape = [t.shape[i] for i in order[:3]] + [t.shape[3] + pad]
    buf = torch.full((start + math.prod(shape),), float("nan"), dtype=t.dtype, device="cuda")
    back = [order.index(i) for i in range(4)]
    out = buf[start:].view(shape)[..., :t.shape[3]].permute(back)
    out.copy_(t)
    return out


LAYOUTS = [("bthd", 0, 0), ("bhtd", 0, 0), ("thbd", 8, 8), ("bthd", 3, 1), ("bhtd", 1, 2)]


def check(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax((np.abs(got - ref) / np.maximum(bound, 1e-300))[bad])),
                           np.argwhere(bad)[:4].tolist())


# ------------------------------------------------------------------- rotary

def rotary_bound(x, ref, freqs, pos, inter, scale, u):
    """θ·2^-51: the product with 1/2π and its constant; π·e: the reduced angle in
    fp32; 6e: sine, cosine (2 ulp), scale, two products and their sum."""
    n = len(freqs)
    th = np.abs(pos[:, :, None, None] * freqs)
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    b = np.zeros(x.shape)
    b[..., one] = b[..., two] = scale * (np.abs(x[..., one]) + np.abs(x[..., two])) * ((math.pi + 6) * E + th * 2.0 ** -51)
    b[..., :2 * n] += u * (np.abs(ref) + b)[..., :2 * n]
    return b


ROTARY = [  # batch, tokens, heads, kv, dim, rotated
    (1, 1, 4, 2, 64, 64), (2, 37, 6, 2, 64, 64), (1, 130, 1, 1, 2, 2), (3, 11, 5, 5, 72, 38), (2, 3, 3, 1, 33, 6),
    (1, 5, 40, 8, 128, 128), (1, 9, 2, 2, 1024, 1024), (1, 2, 3, 0, 1001, 998), (65, 1, 4, 4, 96, 48), (1, 3, 257, 1, 16, 8)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", ROTARY)
def test_rotary(lib, case, inter, dtype):
    batch, tokens, heads, kv, dim, rot = case
    q, k = rand((batch, tokens, heads, dim), 1, dtype), rand((batch, tokens, kv, dim), 2, dtype)
    freqs, scale = 10000.0 ** (-np.arange(rot // 2) * 2.0 / rot), float(np.float32(1.25))
    f = torch.from_numpy(freqs).cuda()
    far = np.random.RandomState(3).randint(-(1 << 31), 1 << 31, (batch, tokens))
    near = np.broadcast_to(np.arange(tokens) + 1000, (batch, tokens))
    for i, (pos, kw) in enumerate(((far, dict(positions=torch.from_numpy(far).cuda())),
                                   (far, dict(positions=torch.from_numpy(far).int().cuda())),
                                   (near, dict(start=1000)), (near, dict(positions=torch.arange(1000, 1000 + tokens).cuda())))):
        layout = LAYOUTS[(i + heads) % len(LAYOUTS)]
        for fn, inverse in ((lib.muon_rotary, False), (lib.muon_rotary_grad, True)):
            gq, gk = fn(place(q, *layout), place(k, *layout), f, interleaved=inter, scale=scale, **kw)
            for got, x in ((gq, f64(q)), (gk, f64(k))):
                ref = oa.rotary(x, freqs, pos, inter, scale, inverse)
                check(got, ref, rotary_bound(x, ref, freqs, pos, inter, scale, UNIT[dtype]), (layout, i, inverse))
                assert np.array_equal(f64(got)[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim,rot,inter", [(64, 64, False), (72, 38, False), (72, 38, True), (33, 32, True)])
def test_rotary_in_place_in_one_projection(lib, dim, rot, inter, dtype):
    """q, k and v side by side, as one product gives them: q and k turn in
    place, v and the gaps keep their bits."""
    both = rand((2, 19, 8, dim), 4, dtype).cuda()
    before = both.clone()
    q, k = both[:, :, :5], both[:, :, 5:7]
    f = torch.from_numpy(100.0 ** (-np.arange(rot // 2) * 2.0 / rot)).cuda()
    want = lib.muon_rotary(q.contiguous(), k.contiguous(), f, interleaved=inter)
    lib.muon_rotary(q, k, f, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(both[:, :, 7], before[:, :, 7])
    assert torch.equal(q[..., rot:], before[:, :, :5, rot:])
    one = before[0, :, None].clone()  # one token of 19 batch entries
    q, k = one[:, :, :5], one[:, :, 5:7]
    pos = torch.arange(19, device="cuda")[:, None]
    lib.muon_rotary(q, k, f, positions=pos, interleaved=inter, q_out=q, k_out=k)
    assert torch.equal(q[:, 0], want[0][0]) and torch.equal(k[:, 0], want[1][0])
    # three dimensions, values apart, an output with gaps
    t = before[0, :, :5].transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.full((19, 5, dim + 3), 7.0, dtype=dtype, device="cuda")
    lib.muon_rotary(t, None, f, interleaved=inter, q_out=out[..., :dim])
    assert torch.equal(out[..., :dim], want[0][0]) and bool((out[..., dim:] == 7).all())


def test_rotary_values(lib):
    """No turn at position 0; a pair of infinities or NaN stays its own; empty
    tensors."""
    x = rand((1, 3, 2, 8), 5, torch.float32).cuda()
    f = torch.from_numpy(10.0 ** -np.arange(4.0)).cuda()
    zero = torch.zeros(3, dtype=torch.int64, device="cuda")
    assert torch.equal(lib.muon_rotary(x, None, f, positions=zero)[0], x)
    bad = x.clone()
    bad[0, 1, 1, 2], bad[0, 2, 0, 7] = float("nan"), float("inf")
    y, ref = lib.muon_rotary(bad, None, f)[0], lib.muon_rotary(x, None, f)[0]
    hit = torch.zeros_like(x, dtype=torch.bool)
    hit[0, 1, 1, [2, 6]] = hit[0, 2, 0, [3, 7]] = True
    assert torch.equal(y[~hit], ref[~hit]) and not torch.isfinite(y[hit]).any()
    for shape in ((0, 3, 2, 8), (2, 0, 2, 8), (2, 3, 0, 8)):
        e = torch.empty(shape, device="cuda")
        assert lib.muon_rotary(e, None, f)[0].shape == shape


# ------------------------------------------------------------------ dropout

DROP = [(1, 1), (1, 3), (7, 5), (64, 64), (33, 1001), (3, 4096), (1000, 1), (2, 100003)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", DROP)
def test_dropout(lib, rows, cols, dtype):
    x, r = rand((rows, cols), 6, dtype), rand((rows, cols), 7, dtype)
    u = UNIT[dtype]
    for pad, p, seed, offset in ((0, 0.1, 1, 0), (0, 0.5, 2 ** 64 - 1, 2 ** 64 - 3), (3, 0.9, 12345678901234, 1 << 40),
                                 (8, 1.0, 3, 4), (1, 0.0, 5, 6), (0, 2.0 ** -34, 7, 8), (2, 1 - 2.0 ** -34, 7, 8)):
        dev = [place(t[None, None], "bthd", pad, pad)[0, 0] for t in (x, r)]
        keep = oa.dropout_keep(rows * cols, p, seed, offset).reshape(rows, cols)
        y = oa.dropout(f64(x), p, seed, offset)
        # 1/(1 − p) in fp32, the product, the sum; then the stored type
        slack = 3 * E * np.abs(y)
        got = lib.muon_dropout(dev[0], p, seed, offset)
        check(got, y, slack + u * np.abs(y) * 1.01, ("dropout", pad, p))
        assert not f64(got)[~keep].any()
        ref = f64(r) + y
        both = lib.muon_dropout(dev[0], p, seed, offset, residual=dev[1])
        check(both, ref, slack + (u + E) * (np.abs(ref) + slack), ("residual", pad, p))
        assert np.array_equal(f64(both)[~keep], f64(r)[~keep])
        assert torch.equal(lib.muon_dropout_grad(dev[0], p, seed, offset), got)
        # the offset from the device, in place, and an output with gaps
        at = torch.tensor([offset - (1 << 64) if offset >= 1 << 63 else offset], device="cuda")
        for out in (dev[0].clone(), place(x[None, None], "bthd", 5, 3)[0, 0]):
            assert torch.equal(lib.muon_dropout(out, p, seed, at, residual=dev[1], out=out), both)
        res = dev[1].clone()
        assert torch.equal(lib.muon_dropout(dev[0], p, seed, at, residual=res, out=res), both)
        buf = torch.full((rows, cols + 2), 7.0, dtype=dtype, device="cuda")
        lib.muon_dropout_grad(dev[0], p, seed, at, out=buf[:, 1:-1])
        assert torch.equal(buf[:, 1:-1], got) and bool((buf[:, [0, -1]] == 7).all())


def test_dropout_values(lib):
    """A dropped infinity or NaN leaves nothing; empty tensors."""
    x = torch.full((4, 1000), float("nan"), device="cuda")
    x[::2] = float("inf")
    keep = torch.from_numpy(oa.dropout_keep(4000, 0.6, 9, 1).reshape(4, 1000)).cuda()
    y = lib.muon_dropout(x, 0.6, 9, 1)
    assert not y[~keep].any() and not torch.isfinite(y[keep]).any()
    assert lib.muon_dropout(x[:0], 0.6, 9).shape == (0, 1000) and lib.muon_dropout(x[:, :0], 0.6, 9).shape == (4, 0)


def test_dropout_past_32_bits(lib):
    """Elements past 2^32 have words of their own (counters past 32 bits are
    reached at 2^34 elements, above a test's memory)."""
    rows, cols, tail = (1 << 12) + 1, 1 << 20, 1 << 20
    x = torch.ones((rows, cols), dtype=torch.bfloat16, device="cuda")
    lib.muon_dropout(x, 0.25, 11, 13, out=x)
    for start in (0, (1 << 32) - tail, 1 << 32):
        keep = oa.dropout_keep(tail, 0.25, 11, 13, start)
        got = x.view(-1)[start:start + tail].cpu().float().numpy()
        assert np.array_equal(got != 0, keep)
        assert np.all(np.abs(got[keep] - 4 / 3) <= 4 / 3 * 2.0 ** -8)


# --------------------------------------------------- differential attention

def attention_inputs(batch, queries, keys, heads, kv, dim, dtype, seed=20):
    return (rand((batch, queries, 2 * heads, dim), seed, dtype), rand((batch, keys, 2 * kv, dim), seed + 1, dtype),
            rand((batch, keys, kv, 2 * dim), seed + 2, dtype), rand((heads,), seed + 3, torch.float32),
            rand((batch, queries, heads, 2 * dim), seed + 4, dtype))


def close(got, ref, tol, what):
    assert np.linalg.norm(f64(got) - ref) <= tol * np.linalg.norm(ref), what


def run_case(lib, ts, causal=True, scale=None, offsets=None, layout=LAYOUTS[0], what=None, rand=True):
    q, k, v, lam, do = ts
    dtype = q.dtype
    dev = [place(t, *layout) for t in (q, k, v, do)]
    off = None
    if offsets is not None:
        off, dev = torch.tensor(offsets, dtype=torch.int32, device="cuda"), [t[0] for t in dev]
    dq_, dk_, dv_, do_ = dev
    kw = dict(causal=causal, scale=scale, offsets=off)
    got, saved = lib.muon_diff_attention(dq_, dk_, dv_, lam.cuda(), save=True, **kw)
    args = [f64(t) for t in (q, k, v, lam)]
    u = UNIT[dtype] if dtype == torch.bfloat16 else E
    ref, bound = oa.diff_attention(*args, causal, scale, offsets, u)
    one = (lambda t: t[None]) if offsets is not None else (lambda t: t)
    check(one(got), ref, bound + TINY, ("out", what))
    slack = 8 * E * (math.sqrt(k.shape[1] + q.shape[1] * q.shape[2] / k.shape[2]) + 16)
    tol = slack + (4 * u if dtype == torch.bfloat16 else 0)
    if rand:
        close(one(got), ref, tol, ("out", what))
    assert torch.equal(got, lib.muon_diff_attention(dq_, dk_, dv_, lam.cuda(), **kw))
    back = lambda: lib.muon_diff_attention_grad(do_, dq_, dk_, dv_, lam.cuda(), got, saved, **kw)
    grads = back()
    refs, errs = oa.diff_attention_grad(f64(do), *args, causal, scale, offsets, u)
    for name, g in zip(("dq", "dk", "dv", "dlam"), grads):
        check(g if name == "dlam" else one(g), refs[name], errs[name] + TINY, (name, what))
        if rand and name != "dlam":
            close(one(g), refs[name], tol, (name, what))
        elif rand:
            check(g, refs[name], 2 * slack * np.sqrt(errs["dlam²"]) + TINY, (name, what))
    assert all(torch.equal(a, b) for a, b in zip(grads, back()))
    return got, grads


ATTENTION = [  # batch, queries, keys, heads, kv heads, dim
    (1, 1, 1, 1, 1, 64), (2, 37, 37, 4, 2, 64), (1, 33, 200, 2, 2, 64), (1, 130, 130, 3, 1, 64), (2, 257, 257, 2, 1, 64),
    (1, 300, 411, 7, 1, 64), (3, 5, 2, 4, 4, 64), (1, 70, 3, 6, 2, 64), (2, 64, 64, 8, 1, 128), (1, 129, 161, 2, 1, 128),
    (1, 5, 2, 6, 3, 128), (1, 45, 45, 2, 2, 1), (1, 97, 97, 2, 1, 5), (2, 40, 66, 3, 3, 17), (1, 100, 100, 4, 2, 72),
    (1, 31, 95, 2, 1, 120), (1, 66, 130, 2, 2, 33), (1, 1, 64, 2, 2, 32), (5, 2, 33, 1, 1, 8), (1, 32, 1, 2, 2, 40),
    (1, 1, 700, 6, 2, 64), (2, 3, 1500, 6, 2, 128), (1, 1, 5000, 28, 4, 64), (4, 1, 1025, 3, 3, 72), (1, 20, 3001, 2, 1, 64)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("case", ATTENTION)
def test_attention(lib, case, causal, dtype):
    ts = attention_inputs(*case, dtype)
    run_case(lib, ts, causal, layout=LAYOUTS[sum(case) % len(LAYOUTS)], scale=None if causal else 0.3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 40, 33])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_attention_layouts(lib, layout, dim, dtype):
    run_case(lib, attention_inputs(2, 50, 70, 4, 2, dim, dtype), layout=layout)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_long(lib, dim, dtype):
    """Blocks of several tiles, dealt out one by one and in stretches."""
    run_case(lib, attention_inputs(1, 1500, 1500, 2, 1, dim, dtype))


PACKED = {
    "plain": (300, [0, 1, 2, 50, 178, 300]), "one": (70, [0, 70]), "gaps": (200, [13, 40, 40, 40, 180]),
    "none": (40, [20, 20]), "outside": (100, [-5, 30, 1 << 30, 60]), "falling": (128, [100, 20, 110, 10]),
    "single tokens": (150, list(range(151))), "more than tokens": (65, [0, 3, 3, 3] + [64] * 2000 + [65]),
    "long and short": (700, [0, 1, 2, 3, 690, 695, 700])}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", PACKED)
def test_attention_packed(lib, name, causal, dtype):
    """Whatever the offsets hold; NaN outside every sequence reaches nothing."""
    tokens, offsets = PACKED[name]
    dim, heads, kv = (64, 3, 1) if len(name) % 2 else (72, 4, 2)
    ts = attention_inputs(1, tokens, tokens, heads, kv, dim, dtype)
    inside = np.zeros(tokens, bool)
    for a, b in oa.spans(tokens, offsets):
        inside[a:b] = True
    for t in (ts[0], ts[1], ts[2], ts[4]):
        t[:, ~torch.from_numpy(inside)] = float("nan")
    nan = [t.clone() for t in ts]
    for t in (ts[0], ts[1], ts[2], ts[4]):  # (the oracle reads the sequences alone; 0 keeps its sums finite)
        t[:, ~torch.from_numpy(inside)] = 0.0
    got, grads = run_case(lib, ts, causal, offsets=offsets, what=name)
    dev = [t[0].cuda() for t in (nan[0], nan[1], nan[2])] + [nan[3].cuda()]
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    out, saved = lib.muon_diff_attention(*dev, causal=causal, offsets=off, save=True)
    assert torch.equal(out, got) and not out[~torch.from_numpy(inside).cuda()].any()
    again = lib.muon_diff_attention_grad(nan[4][0].cuda(), *dev, out, saved, causal=causal, offsets=off)
    assert all(torch.equal(a, b) for a, b in zip(again, grads))
    for t in grads[:3]:
        assert not t[~torch.from_numpy(inside).cuda()].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kind", ["rising", "falling", "spike", "flat", "far below"])
def test_attention_scores(lib, kind, dim, dtype):
    """Maxima that grow with every key, late, or never; a softmax of one key;
    scores of ±thousands."""
    n = 200
    ts = list(attention_inputs(1, 40, n, 2, 1, dim, dtype))
    q, k = (torch.zeros_like(t) for t in ts[:2])
    q[..., 0] = 1.0
    x = torch.arange(n, dtype=torch.float64)
    x = {"rising": 4 * x, "falling": -4 * x, "spike": 900.0 * (x == 170), "flat": 0 * x + 3000, "far below": 0 * x - 5000}[kind]
    k[0, :, :, 0] = x.to(dtype)[:, None]
    k[0, :, :, 1:3] = rand((n, 2, 2), 33, dtype)
    q[..., 1:3] = rand(tuple(q.shape[:3]) + (2,), 34, dtype)
    ts[:2] = q, k
    run_case(lib, ts, True, scale=1.0, what=kind, rand=False)
    run_case(lib, ts, False, scale=0.5, what=kind, rand=False)


@pytest.mark.parametrize("power", [-100, -40, 40, 60])
@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_magnitudes(lib, power, dtype):
    """Values and gradients of any size: errors stay relative to the terms (the
    products of both stay above 2^-126 and below 2^128)."""
    q, k, v, lam, do = attention_inputs(1, 75, 75, 2, 1, 64, dtype)
    run_case(lib, (q, k, v * 2.0 ** power, lam, do * 2.0 ** (20 if power < 0 else 0)))


@pytest.mark.parametrize("power", [-60, 60])
@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_scales(lib, power, dtype):
    """The smallest and largest scale, with scores of ordinary size from them."""
    q, k, v, lam, do = attention_inputs(1, 75, 75, 2, 1, 64, dtype)
    run_case(lib, (q * 2.0 ** -(power // 2), k * 2.0 ** -(power // 2), v, lam, do), scale=2.0 ** power)
    if power < 0:  # flat maps: scores that all but vanish
        run_case(lib, (q, k, v, lam, do), scale=2.0 ** power)


@pytest.mark.parametrize("lam", [0.0, 1.0, -3.0, 100.0])
@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_lambda(lib, lam, dtype):
    ts = list(attention_inputs(1, 60, 60, 2, 1, 64, dtype))
    ts[3] = torch.tensor([lam, 0.5])
    run_case(lib, ts)


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_same_maps_cancel(lib, dtype):
    """With equal maps and λ = 1 nothing is left, and λ's gradient stays."""
    q, k, v, lam, do = attention_inputs(1, 90, 90, 2, 1, 64, dtype)
    q[:, :, 1::2], k[:, :, 1::2] = q[:, :, ::2], k[:, :, ::2]
    got, _ = run_case(lib, (q, k, v, torch.ones(2), do), rand=False)
    assert not got.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_hidden_keys(lib, dtype):
    """Keys that no row sees (more keys than queries never has these; keys of
    later rows do): infinities and NaN in k there change no earlier row."""
    q, k, v, lam, _ = (t.cuda() for t in attention_inputs(1, 100, 100, 2, 1, 64, dtype))
    ref = lib.muon_diff_attention(q, k, v, lam)
    k[:, 60:70], k[:, 70:] = float("nan"), float("inf")
    got = lib.muon_diff_attention(q, k, v, lam)
    assert torch.equal(got[:, :60], ref[:, :60]) and not torch.isfinite(got[:, 60:]).any()
    one = lib.muon_diff_attention(q, k, v, lam, causal=False)
    assert not torch.isfinite(one).any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_attention_bad_rows_stay_alone(lib, dtype):
    """A NaN in a query, or in a head, reaches no other row or group."""
    q, k, v, lam, _ = (t.cuda() for t in attention_inputs(2, 70, 70, 4, 2, 64, dtype))
    ref = lib.muon_diff_attention(q, k, v, lam)
    q[0, 33, 2] = float("nan")  # head 1
    v[1, :, 1, 5] = float("inf")  # heads 2 and 3, value 5
    got = lib.muon_diff_attention(q, k, v, lam)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[0, 33, 1] = True
    hit[1, :, 2:, 5] = True
    assert torch.equal(got[~hit], ref[~hit]) and not torch.isfinite(got[hit]).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("case", [(1, 0, 5, 2, 1, 64), (0, 5, 5, 2, 1, 64), (1, 5, 0, 2, 1, 64), (2, 70, 0, 4, 2, 72),
                                  (2, 1, 0, 2, 2, 128), (1, 0, 0, 1, 1, 8)])
def test_attention_empty(lib, case, dtype):
    """No queries, no keys: zeros, and gradients of zero."""
    q, k, v, lam, do = (t.cuda() for t in attention_inputs(*case, dtype))
    for causal in (True, False):
        out, saved = lib.muon_diff_attention(q, k, v, lam, causal=causal, save=True)
        assert out.shape == do.shape and not out.any()
        grads = lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved, causal=causal)
        assert [g.shape for g in grads] == [q.shape, k.shape, v.shape, lam.shape] and not any(g.any() for g in grads)


def test_attention_wanted_gradients(lib):
    """Each gradient alone has the bits it has among the others, in outputs of
    any strides."""
    import ctypes
    from muon_newton_schulz_06_amd import attention
    q, k, v, lam, do = (t.cuda() for t in attention_inputs(2, 70, 90, 4, 2, 40, torch.bfloat16))
    out, saved = lib.muon_diff_attention(q, k, v, lam, save=True)
    ref = lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved)
    for i, kw in ((0, dict(want_dkv=False, want_dlam=False)), (1, dict(want_dq=False, want_dlam=False)),
                  (3, dict(want_dq=False, want_dkv=False))):
        one = lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved, **kw)
        assert torch.equal(one[i], ref[i])
        assert [t is None for t in one] == [j != i and not (i == 1 and j == 2) for j in range(4)]
    L = attention._lib()
    f, kept = attention._attention(q, k, v, lam, True, None, None)
    for layout in LAYOUTS:
        gq, gk, gv = (place(torch.zeros(t.shape, dtype=t.dtype), *layout) for t in (q, k, v))
        st = [attention._strides(t) for t in (gq, gk, gv)]
        g = attention.MuonDiffAttentionGrads(gq.data_ptr(), gk.data_ptr(), gv.data_ptr(), None, *st)
        n, ds = ctypes.c_size_t(0), attention._strides(do)
        assert L.muon_diff_attention_workspace_size(ctypes.byref(f), do.data_ptr(), ds, ctypes.byref(n)) == 0
        ws = torch.empty(n.value, dtype=torch.uint8, device="cuda")
        assert L.muon_diff_attention_grad(ctypes.byref(f), do.data_ptr(), ds, out.data_ptr(), ds, saved.data_ptr(),
                                          saved.numel(), ctypes.byref(g), ws.data_ptr(), n.value,
                                          torch.cuda.current_stream().cuda_stream) == 0
        for a, b, t in ((gq, ref[0], q), (gk, ref[1], k), (gv, ref[2], v)):
            assert torch.equal(a, b)
            _, pad, start = layout
            base = torch.as_strided(a, (start,), (1,), 0)
            assert bool(torch.isnan(base).all())  # what lies in front is left alone
    got = place(torch.zeros(out.shape, dtype=out.dtype), "bhtd", 3, 1)
    lib.muon_diff_attention(q, k, v, lam, out=got)
    assert torch.equal(got, out)


def test_gradients_by_differences(lib):
    """The kernels' gradients along random directions against central
    differences of the fp64 formula: its third derivatives leave about ε²."""
    q, k, v, lam, do = attention_inputs(1, 40, 50, 4, 2, 64, torch.float32)
    args, w = [f64(t) for t in (q, k, v, lam)], f64(do)
    out, saved = lib.muon_diff_attention(*(t.cuda() for t in (q, k, v, lam)), save=True)
    grads = lib.muon_diff_attention_grad(do.cuda(), *(t.cuda() for t in (q, k, v, lam)), out, saved)
    _, errs = oa.diff_attention_grad(w, *args, unit=E)
    r, eps = np.random.RandomState(7), 1e-4
    for i, name in enumerate(("dq", "dk", "dv", "dlam")):
        d = r.randn(*args[i].shape)
        f = [(oa.diff_attention(*args[:i], args[i] + s * d, *args[i + 1:])[0] * w).sum() for s in (eps, -eps)]
        want, got = (f[0] - f[1]) / (2 * eps), (f64(grads[i]) * d).sum()
        assert abs(got - want) <= (errs[name] * np.abs(d)).sum() + 1e-6 * np.abs(w).sum(), name
    x, freqs, pos = f64(q), 100.0 ** (-np.arange(32) / 32.0), np.arange(40)[None]
    dy = rand(q.shape, 40, torch.float32)
    dx, _ = lib.muon_rotary_grad(dy.cuda(), None, torch.from_numpy(freqs).cuda())
    d = r.randn(*x.shape)  # (linear: the difference is exact)
    want = ((oa.rotary(x + d, freqs, pos) - oa.rotary(x, freqs, pos)) * f64(dy)).sum()
    assert abs((f64(dx) * d).sum() - want) <= 12 * E * 2 * (np.abs(f64(dy)).sum() + 1) * np.abs(d).max()


# ------------------------------------------------------------------ together

def leaf(shape, seed, dtype=torch.float32, std=1.0):
    return rand(shape, seed, dtype, std).cuda().requires_grad_()


def test_modules_match_functions(lib):
    """Autograd through the modules gives the functions' bits, for broadcast and
    transposed incoming gradients too, and nothing is computed without need."""
    q, k, v = (leaf(s, i, torch.bfloat16) for i, s in enumerate(((2, 33, 8, 32), (2, 33, 4, 32), (2, 33, 2, 64))))
    rot = lib.Rotary(32, 16, scaling="linear", factor=2.0)
    a, b = rot(q, k)
    (a.sum() + (b.transpose(1, 2) * 2).sum()).backward()
    f = rot.freqs.cuda()
    ra, rb = lib.muon_rotary(q.detach(), k.detach(), f)
    assert torch.equal(a, ra) and torch.equal(b, rb)
    ga, gb = lib.muon_rotary_grad(torch.ones_like(ra), torch.full_like(rb, 2), f)
    assert torch.equal(q.grad, ga) and torch.equal(k.grad, gb)
    k.grad = q.grad = None
    rot(q, k, start=3)[1].sum().backward()  # one of the two alone
    assert k.grad is not None and (q.grad is None or not q.grad.any())
    assert torch.equal(rot(q.detach()), rot(q.detach(), k.detach())[0])
    q.grad = k.grad = None
    att = lib.DiffAttention(4, 32, 2, device="cuda", dtype=torch.bfloat16)
    y = att(q, k, v)
    w = rand(tuple(y.shape), 9, torch.bfloat16).cuda().transpose(1, 2).contiguous().transpose(1, 2)
    (y * w).sum().backward()
    lam = att.lam().detach().contiguous()
    out, saved = lib.muon_diff_attention(q.detach(), k.detach(), v.detach(), lam, save=True)
    gain = (att.weight * (1 - att.lambda_init)).detach()
    n, _, rstd = lib.muon_rms_norm(out, gain, eps=1e-5)
    assert torch.equal(y, n)
    do, dw = lib.muon_rms_norm_grad(w, out, gain, rstd)
    grads = lib.muon_diff_attention_grad(do, q.detach(), k.detach(), v.detach(), lam, out, saved)
    assert all(torch.equal(t.grad, g) for t, g in zip((q, k, v), grads))
    one = (att.lambda_q1 @ att.lambda_k1).exp().detach()
    assert torch.allclose(att.lambda_q1.grad, grads[3].sum() * one * att.lambda_k1.detach(), rtol=1e-5, atol=1e-7)
    with torch.no_grad():
        assert torch.equal(att(q, k, v), y)
    # frozen tensors get no gradients
    v2 = v.detach()
    q.grad = k.grad = None
    att(q.detach(), k, v2).sum().backward()
    assert q.grad is None and k.grad is not None


def test_dropout_module(lib):
    x, r = leaf((5, 7, 12), 1), leaf((5, 7, 12), 2)
    m = lib.Dropout(0.4, seed=17, device="cuda")
    for call in range(3):
        x.grad = r.grad = None
        y = m(x, r)
        keep = torch.from_numpy(oa.dropout_keep(x.numel(), 0.4, 17, call)).view_as(x).cuda()
        assert torch.equal(y, lib.muon_dropout(x.detach(), 0.4, 17, call, residual=r.detach()))
        y.sum().backward()
        assert torch.equal(x.grad != 0, keep) and bool((r.grad == 1).all())
    assert int(m.calls) == 3 and int(lib.Dropout(0.4)._buffers["calls"]) == 0
    m.load_state_dict(m.state_dict())


def block(lib, x, p, rot, att, drop, norms, ffn, offsets=None):
    """A block of a decoder: attention and feed-forward halves with dropout."""
    t = (*x.shape[:-1], -1)
    n = norms[0](x)
    q, k, v = (n @ p["qk"]).view(*x.shape[:-1], 12, 32), None, (n @ p["v"]).view(*x.shape[:-1], 2, 64)
    q, k = rot(q[..., :8, :], q[..., 8:, :])
    x = drop(att(q, k, v, offsets).reshape(t) @ p["o"], x)
    return drop(ffn(norms[1](x)), x)


def make_block(lib, dtype, dim=96):
    torch.manual_seed(3)
    p = {n: leaf(s, 50 + i, dtype, s[0] ** -0.5) for i, (n, s) in enumerate(
        (("qk", (dim, 12 * 32)), ("v", (dim, 128)), ("o", (4 * 64, dim))))}
    kw = dict(device="cuda", dtype=dtype)
    return (p, lib.Rotary(32), lib.DiffAttention(4, 32, 2, **kw), lib.Dropout(0.2, seed=5, device="cuda"),
            [lib.RMSNorm(dim, **kw) for _ in range(2)], lib.GatedFFN(dim, 160, **kw))


def block_parameters(parts):
    p, _, att, _, norms, ffn = parts
    return [*p.values(), *att.parameters(), *(w for n in norms for w in n.parameters()), *ffn.parameters()]


def test_block_gradients(lib):
    """A whole block's gradients against differences of its own fp32 forward
    pass: a step ε along a direction of unit length changes the loss by its
    derivative times 2ε, up to the fp32 rounding of two losses and ε² of the
    third derivative."""
    parts = make_block(lib, torch.float32)
    x, w = leaf((2, 21, 96), 70), rand((2, 21, 96), 71, torch.float32).cuda()
    leaves = [x, *block_parameters(parts)]

    def loss():
        parts[3].calls.zero_()
        return (block(lib, x, *parts).double() * w).sum()
    loss().backward()
    for i, t in enumerate(leaves):
        assert t.grad is not None and torch.isfinite(t.grad).all()
        d = torch.nn.functional.normalize(rand(tuple(t.shape), 80 + i, torch.float32).cuda().flatten(), dim=0).view_as(t)
        f = {}
        for eps in (2.0 ** -5, 2.0 ** -6):  # (halved: a quarter of what the third derivative leaves)
            with torch.no_grad():
                keep = t.detach().clone()
                t.add_(d, alpha=eps)
                a = loss()
                t.copy_(keep).add_(d, alpha=-eps)
                b = loss()
                t.copy_(keep)
            f[eps] = float(a - b) / (2 * eps)
        want, got = (4 * f[2.0 ** -6] - f[2.0 ** -5]) / 3, float((t.grad.double() * d).sum())
        # each of some 4000 results is off by some hundred roundings of its size
        # (about 2) in either loss; times |w| about 1, random signs: their sum by
        # 64·100·2·2^-24 < 1e-3, over 2ε = 2^-5: 0.03, times 5/3
        assert abs(got - want) <= 0.05 + 0.02 * abs(want), (i, got, want)


@pytest.mark.parametrize("dtype", DTYPES)
def test_block_packed_is_its_sequences(lib, dtype):
    """A packed batch of the whole block gives what its sequences give alone (no
    dropping: its draws go by the place in the batch)."""
    parts = make_block(lib, dtype)
    parts[3].eval()
    x = rand((50, 96), 72, dtype).cuda()
    off = torch.tensor([0, 20, 21, 50], dtype=torch.int32, device="cuda")
    pos = torch.cat([torch.arange(n) for n in (20, 1, 29)]).cuda()

    class At(torch.nn.Module):
        def forward(self, q, k):
            q, k = parts[1](q[None], k[None], positions=pos)
            return q[0], k[0]
    with torch.no_grad():
        both = block(lib, x, parts[0], At(), *parts[2:], off)
        for a, b in ((0, 20), (20, 21), (21, 50)):
            one = block(lib, x[None, a:b], *parts)[0]
            # other tiles, other orders of the fp32 sums: a bf16 result may round the
            # other way now and then, and what follows sees that
            tol = 8 * UNIT[dtype] if dtype == torch.bfloat16 else 2000 * E
            assert float((both[a:b] - one).abs().max()) <= tol * float(one.abs().max())


def test_other_stream_and_graph(lib):
    """The same bits on another stream, through `stream`, and from a replayed
    graph with eager work between the replays."""
    q, k, v, lam, do = (t.cuda() for t in attention_inputs(2, 150, 150, 4, 2, 64, torch.bfloat16))
    q1, k1, v1 = (t.cuda() for t in attention_inputs(1, 1, 3000, 4, 2, 64, torch.bfloat16)[:3])
    off = torch.tensor([0, 100, 290, 300], dtype=torch.int32, device="cuda")
    f = torch.from_numpy(10.0 ** (-np.arange(32) / 8.0)).cuda()
    at = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        a, b = lib.muon_rotary(q, k, f)
        o, s = lib.muon_diff_attention(a, b, v, lam, save=True)
        g = lib.muon_diff_attention_grad(do, a, b, v, lam, o, s)
        one = lib.muon_diff_attention(q1, k1, v1, lam)
        flat = [t.flatten(0, 1) for t in (q, k, v)]
        p, ps = lib.muon_diff_attention(*flat, lam, offsets=off, save=True)
        pg = lib.muon_diff_attention_grad(do.flatten(0, 1), *flat, lam, p, ps, offsets=off)
        d = lib.muon_dropout(o, 0.3, 5, at, residual=do)
        odd = lib.muon_diff_attention(q[..., :33], k[..., :33], v[..., :66], lam)
        return [a, b, o, *g, one, p, *pg, d, lib.muon_dropout_grad(do, 0.3, 5, at), *lib.muon_rotary_grad(a, b, f), odd]
    ref = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    side.wait_stream(torch.cuda.current_stream())
    vt = v.transpose(2, 3).contiguous().transpose(2, 3)  # copied, on that stream
    y, ro = lib.muon_diff_attention(ref[0], ref[1], vt, lam, stream=side), lib.muon_rotary(q, k, f, stream=side)
    dr = lib.muon_dropout(ref[2], 0.3, 5, at, residual=do, stream=side)
    side.synchronize()
    assert torch.equal(y, ref[2]) and torch.equal(ro[0], ref[0]) and torch.equal(dr, ref[13])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        for t in outs:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, outs))
        step()
    at.fill_(2)  # the draws of a replay follow the counter
    graph.replay()
    assert torch.equal(outs[13], lib.muon_dropout(ref[2], 0.3, 5, 2, residual=do)) and not torch.equal(outs[13], ref[13])


def test_captured_training_block(lib):
    """A block's forward and backward pass in a graph, its dropout drawing anew
    each replay: the gradients of as many eager passes."""
    parts = make_block(lib, torch.bfloat16)
    x, w = rand((2, 40, 96), 73, torch.bfloat16).cuda(), rand((2, 40, 96), 74, torch.bfloat16).cuda()
    leaves = block_parameters(parts)

    def step():
        grads = torch.autograd.grad(block(lib, x, *parts), leaves, w)
        return [g.detach() for g in grads]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    parts[3].calls.zero_()
    eager = [[g.clone() for g in step()] for _ in range(3)]
    parts[3].calls.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    parts[3].calls.zero_()
    for ref in eager:
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, outs))
        rand((64, 64), 1, torch.float32).cuda() @ torch.ones(64, 64, device="cuda")
    assert not torch.equal(eager[0][0], eager[1][0])


def test_workspaces(lib):
    """A buffer of the caller's of the size asked for; one too small is refused."""
    for ts in (attention_inputs(1, 1, 3000, 4, 2, 64, torch.bfloat16), attention_inputs(2, 70, 70, 4, 2, 33, torch.float32)):
        q, k, v, lam, do = (t.cuda() for t in ts)
        b, nq, h2, dim = q.shape
        sizes = (b, nq, k.shape[1], h2 // 2, k.shape[2] // 2, dim, q.dtype)
        ref, saved = lib.muon_diff_attention(q, k, v, lam, save=True)
        assert saved.numel() == lib.diff_attention_saved_size(*sizes)
        gref = lib.muon_diff_attention_grad(do, q, k, v, lam, ref, saved)
        n, m = lib.diff_attention_workspace_size(*sizes), lib.diff_attention_workspace_size(*sizes, grad=True)
        ws = torch.full((max(n, m),), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(lib.muon_diff_attention(q, k, v, lam, workspace=ws[:n]), ref)
        ws.fill_(255)
        got = lib.muon_diff_attention_grad(do, q, k, v, lam, ref, saved, workspace=ws[:m])
        assert all(torch.equal(a, c) for a, c in zip(got, gref))
        with pytest.raises(lib.MuonError):
            lib.muon_diff_attention_grad(do, q, k, v, lam, ref, saved, workspace=ws[:256])
        with pytest.raises(lib.MuonError):
            lib.muon_diff_attention_grad(do, q, k, v, lam, ref, saved[:256])


def test_example_runs(lib):
    """The example takes a few steps; its gradients are finite and reach every
    parameter."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_attention_lm.py")
    spec = importlib.util.spec_from_file_location("train_attention_lm", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.train(steps=3, tokens=300, documents=4, vocab=64, heads=2, kv_heads=1, dim=32, hidden=96, depth=2,
                      log=lambda s: None)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
    net = ex.Model(64, 2, 1, 32, 96, 2, dropout=0.1, device="cuda", dtype=torch.bfloat16)
    ids, offsets, positions = ex.batch(300, 4, 64, torch.Generator(device="cuda").manual_seed(1), "cuda")
    net(ids, offsets, positions).float().square().mean().backward()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() and p.grad.abs().max() > 0 for p in net.parameters())
