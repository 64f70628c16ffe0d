"""Embedding, RMS norm and gated FFN kernels against the fp64 oracle.

Tolerances are element-wise bounds derived from the arithmetic.  u is the unit
roundoff of the stored type (2^-8 bf16, 8 significant bits; 2^-24 fp32), e = 2^-24 that of the
fp32 arithmetic.  A sum of n terms t_k in fp32, in any order, is within
1.01·n·e·Σ|t_k|; a value rounded to the stored type within u of itself; where an
operand of a product was rounded, the product's error is bounded by the same
product of absolute values.
"""
import numpy as np
import pytest
import torch

import oracle.layers as ol

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
UNIT = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}
TINY = 2.0 ** -126
DTYPES = [torch.bfloat16, torch.float32]


def rand(shape, seed, dtype, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g, dtype=torch.float64) * std).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def strided(t, pad):
    """The same 2-D values on the GPU with `pad` extra elements per row and a
    start `pad` elements into the allocation (pad odd: misaligned rows).  The
    gaps hold NaN: reading one shows."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    out = buf[:, pad:]
    out.copy_(t)
    return out


def check(got, ref, bound, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - ref)[bad])),
                           np.argwhere(bad)[:4].tolist())


# ---------------------------------------------------------------- embedding

IDS = [(1, 40, 64), (7, 33, 17), (130, 50, 128), (1000, 300, 129), (1025, 300, 1024), (4097, 900, 40)]


def make_ids(tokens, vocab, seed, dtype, skew=True):
    r = np.random.RandomState(seed)
    ids = r.randint(0, vocab, tokens)
    if skew and tokens > 4:  # one id holds most of the batch, some tokens are padding
        ids[r.rand(tokens) < 0.5] = vocab // 3
        ids[r.rand(tokens) < 0.1] = -1
        ids[r.randint(tokens)] = vocab  # just outside
        ids[r.randint(tokens)] = 0
        ids[r.randint(tokens)] = vocab - 1
    return torch.from_numpy(ids).to(dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("idt", [torch.int64, torch.int32])
@pytest.mark.parametrize("tokens,vocab,dim", IDS)
def test_embedding(lib, tokens, vocab, dim, dtype, idt):
    ids, w = make_ids(tokens, vocab, 1, idt), rand((vocab, dim), 2, dtype)
    scale = float(np.float32(1.7))
    ref = ol.embedding(ids.numpy(), f64(w), scale)
    for pad in (0, 3, 8):
        got = lib.muon_embedding(ids.cuda(), strided(w, pad), scale)
        check(got, ref, (UNIT[dtype] + E) * 1.01 * np.abs(ref) + TINY, ("embedding", pad))


@pytest.mark.parametrize("dtype,gdt", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                       (torch.float32, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("tokens,vocab,dim", IDS)
def test_embedding_grad(lib, tokens, vocab, dim, dtype, gdt):
    ids, dy = make_ids(tokens, vocab, 3, torch.int64), rand((tokens, dim), 4, dtype)
    scale = float(np.float32(0.3))
    ref, mag, n = ol.embedding_grad(f64(dy), ids.numpy(), vocab, scale)
    bound = UNIT[gdt] * np.abs(ref) * 1.01 + 1.01 * (n[:, None] + 2) * E * mag + TINY
    for pad in (0, 3, 4, 8):
        d = strided(dy, pad)
        got = lib.muon_embedding_grad(d, ids.cuda(), vocab, scale, dtype=gdt)
        check(got, ref, bound, ("embedding grad", pad))
        assert torch.equal(got, lib.muon_embedding_grad(d, ids.cuda(), vocab, scale, dtype=gdt))
        # into a strided output, added to what it holds; untouched rows keep their bits
        old = rand((vocab, dim), 5, gdt)
        out = strided(old, pad)
        lib.muon_embedding_grad(d, ids.cuda(), vocab, scale, out=out, accumulate=True)
        check(out, f64(old) + ref, UNIT[gdt] * np.abs(f64(old) + ref) * 1.01
              + 1.01 * (n[:, None] + 3) * E * (mag + np.abs(f64(old))) + TINY, ("accumulate", pad))
        keep = torch.from_numpy(n == 0)
        assert torch.equal(out.cpu()[keep], old[keep])
        gaps = out.as_strided((vocab, pad), (dim + pad, 1), 0) if pad else None
        assert gaps is None or torch.isnan(gaps).all()


@pytest.mark.parametrize("tokens,vocab,dim", [(20000, 700, 24), (40000, 70000, 8), (66000, 3, 16)])
def test_embedding_grad_long(lib, tokens, vocab, dim):
    """Batches sorted in device memory (above 16384 tokens), one to three
    digit passes, runs of tens of thousands of equal ids."""
    ids, dy = make_ids(tokens, vocab, 6, torch.int64), rand((tokens, dim), 7, torch.float32)
    ref, mag, n = ol.embedding_grad(f64(dy), ids.numpy(), vocab, 1.0)
    got = lib.muon_embedding_grad(dy.cuda(), ids.cuda(), vocab)
    check(got, ref, UNIT[torch.float32] * np.abs(ref) + 1.01 * (n[:, None] + 2) * E * mag + TINY, "long")
    assert torch.equal(got, lib.muon_embedding_grad(dy.cuda(), ids.cuda(), vocab))


@pytest.mark.parametrize("tokens", [16383, 16384, 16385])
def test_embedding_grad_sort_limit(lib, tokens):
    """Both sides of the one-workgroup sort's limit, every id distinct or all
    equal: whole numbers, so the sums are exact."""
    dy = torch.arange(tokens * 4, dtype=torch.float32).reshape(tokens, 4) % 17
    perm = torch.randperm(tokens, generator=torch.Generator().manual_seed(3))
    got = lib.muon_embedding_grad(dy.cuda(), perm.cuda(), tokens).cpu()
    ref = torch.empty_like(dy)
    ref[perm] = dy
    assert torch.equal(got, ref)
    same = lib.muon_embedding_grad(dy.cuda(), torch.full((tokens,), 5, device="cuda"), 9).cpu()
    assert torch.equal(same[5], dy.sum(0)) and same.abs().sum(1).nonzero().numel() == 1


def test_embedding_empty(lib):
    w = rand((5, 8), 1, torch.float32).cuda()
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert lib.muon_embedding(none, w).shape == (0, 8)
    dw = torch.full((5, 8), 3.0, device="cuda")
    lib.muon_embedding_grad(torch.empty((0, 8), device="cuda"), none, 5, out=dw, accumulate=True)
    assert (dw == 3).all()
    lib.muon_embedding_grad(torch.empty((0, 8), device="cuda"), none, 5, out=dw)
    assert (dw == 0).all()
    ids = torch.full((4,), -1, device="cuda")  # nothing but padding
    assert (lib.muon_embedding_grad(torch.ones((4, 8), device="cuda"), ids, 5) == 0).all()
    assert (lib.muon_embedding(ids, torch.full((5, 8), float("inf"), device="cuda")) == 0).all()


def test_embedding_masked_places(lib):
    """NaN and infinity where the id is padding, or in rows no token names,
    reach nothing."""
    ids = make_ids(500, 60, 9, torch.int64)
    ids[ids == 7] = 8
    off = (ids < 0) | (ids >= 60)
    w, dy = rand((60, 24), 1, torch.bfloat16), rand((500, 24), 2, torch.bfloat16)
    clean = lib.muon_embedding_grad(torch.where(off[:, None], 0, dy).cuda(), ids.cuda(), 60)
    dy[off] = float("nan")
    w[7] = float("inf")
    assert torch.isfinite(lib.muon_embedding(ids.cuda(), w.cuda())).all()
    assert torch.equal(lib.muon_embedding_grad(dy.cuda(), ids.cuda(), 60), clean)
    assert (clean[7] == 0).all()


# ----------------------------------------------------------------- RMS norm

NORMS = [(1, 1), (1, 3584), (3, 17), (5, 512), (300, 1001), (2100, 96), (2048, 1001), (2500, 4096), (9, 8200),
         (3, 33000), (2, 70000)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim", NORMS)
def test_rms_norm(lib, tokens, dim, dtype):
    x, r = rand((tokens, dim), 1, dtype, 3.0), rand((tokens, dim), 2, dtype)
    u = UNIT[dtype]
    for res in (True, False):
        for wdt in (dtype, torch.float32):
            w = rand((dim,), 3, wdt)
            eps = float(np.float32(1e-5))
            y0, s0, r0 = ol.rms_norm(f64(x), f64(w), f64(r) if res else None, eps)
            for pad in (0, 3):
                y, s, rstd = lib.muon_rms_norm(strided(x, pad), w.cuda(), strided(r, pad) if res else None, eps)
                # relative error of rstd: half that of the mean (dim + 3 roundings of
                # positive terms, s² twice that of s), then the root and the quotient
                er = 0.505 * (dim + 8) * E + 3 * E
                check(rstd, r0, er * r0, "rstd")
                # s may cancel: its rounding is relative to s itself (one fp32 addition)
                check(y, y0, (u + er + 5 * E) * 1.01 * np.abs(y0) + TINY, ("y", pad))
                if res:
                    check(s, s0, (u + E) * 1.01 * np.abs(s0) + TINY, ("s", pad))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,dim", NORMS)
def test_rms_norm_grad(lib, tokens, dim, dtype):
    dy, s, ds = (rand((tokens, dim), k, dtype) for k in (4, 5, 6))
    u = UNIT[dtype]
    for wdt in (dtype, torch.float32):
        w = rand((dim,), 7, wdt)
        rstd = (1.0 / torch.sqrt(s.double().square().mean(1) + 1e-6)).float()
        a, b, c, r64 = f64(dy), f64(s), f64(w), f64(rstd)[:, None]
        for extra in (None, ds):
            dx0, dw0 = ol.rms_norm_grad(a, b, c, f64(rstd), f64(extra) if extra is not None else None)
            n = np.abs(b) * r64
            dots = np.mean(np.abs(c * a) * n, axis=1, keepdims=True)
            bx = u * np.abs(dx0) + 1.01 * E * (r64 * (6 * np.abs(c * a) + (dim + 10) * n * dots)
                                               + 3 * np.abs(dx0)) + TINY
            bw = UNIT[wdt] * np.abs(dw0) + 1.01 * (tokens + 3) * E * (np.abs(a) * n).sum(0) + TINY
            for pad in (0, 3):
                args = (strided(dy, pad), strided(s, pad), w.cuda(), rstd.cuda())
                d = strided(extra, pad) if extra is not None else None
                dx, dw = lib.muon_rms_norm_grad(*args, dsum=d)
                check(dx, dx0, bx * 1.01, ("dx", pad))
                check(dw, dw0, bw * 1.01, ("dweight", pad))
                dx2, dw2 = lib.muon_rms_norm_grad(*args, dsum=d)
                assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
                old = rand((dim,), 8, wdt)
                acc = old.cuda()
                lib.muon_rms_norm_grad(*args, dsum=d, dweight=acc, accumulate=True)
                check(acc, dw0 + f64(old), 1.01 * (bw + UNIT[wdt] * np.abs(dw0 + f64(old))
                                                   + E * np.abs(f64(old))), ("accumulated", pad))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [96, 1001, 33000])
def test_rms_norm_in_place(lib, dim, dtype):
    x, r, w = rand((6, dim), 1, dtype).cuda(), rand((6, dim), 2, dtype).cuda(), rand((dim,), 3, dtype).cuda()
    y, s, rstd = lib.muon_rms_norm(x, w, r)
    x2, r2 = x.clone(), r.clone()
    y2, s2, _ = lib.muon_rms_norm(x2, w, r2, out=x2, sum_out=r2)
    assert y2 is x2 and s2 is r2 and torch.equal(x2, y) and torch.equal(r2, s)
    dy, ds = rand((6, dim), 4, dtype).cuda(), rand((6, dim), 5, dtype).cuda()
    dx, dw = lib.muon_rms_norm_grad(dy, s, w, rstd, dsum=ds)
    dy2, ds2 = dy.clone(), ds.clone()
    assert torch.equal(lib.muon_rms_norm_grad(dy2, s, w, rstd, dsum=ds, out=dy2)[0], dx)
    assert torch.equal(lib.muon_rms_norm_grad(dy, s, w, rstd, dsum=ds2, out=ds2)[0], dx)


def test_rms_norm_values(lib):
    """Zero rows, infinities and NaN stay in their own row; zero tokens."""
    x = rand((5, 64), 1, torch.float32)
    x[1] = 0
    x[2, 3] = float("nan")
    x[3, 3] = float("inf")
    w = torch.ones(64)
    y, _, rstd = lib.muon_rms_norm(x.cuda(), w.cuda())
    y = y.cpu()
    assert torch.isfinite(y[[0, 1, 4]]).all() and (y[1] == 0).all()
    assert torch.isnan(y[2]).all()
    assert torch.isnan(y[3, 3]) and (y[3, :3] == 0).all()
    e = torch.empty((0, 64), device="cuda")
    y, _, rstd = lib.muon_rms_norm(e, w.cuda())
    assert y.shape == (0, 64) and rstd.shape == (0,)
    dx, dw = lib.muon_rms_norm_grad(e, e, w.cuda(), rstd)
    assert dx.shape == (0, 64) and (dw == 0).all()


# -------------------------------------------------- gated feed-forward block

FFNS = [(1, 1, 1), (1, 64, 96), (3, 17, 33), (16, 256, 512), (17, 250, 130), (50, 128, 1000), (65, 512, 264),
        (130, 300, 700), (257, 264, 520), (300, 72, 200)]


def ffn_inputs(tokens, model, hidden, dtype, seed=10):
    return (rand((tokens, model), seed, dtype), rand((hidden, model), seed + 1, dtype, model ** -0.5),
            rand((hidden, model), seed + 2, dtype, model ** -0.5),
            rand((model, hidden), seed + 3, dtype, hidden ** -0.5), rand((tokens, model), seed + 4, dtype))


def ffn_bounds(x, wg, wu, wd, dy, act, dtype, gdt):
    """(results, element-wise error bounds of them), numpy."""
    f = ol.gated_ffn_grad(dy, x, wg, wu, wd, act)
    return f, ffn_errors(f, x, wg, wu, wd, dy, dtype, gdt)


def ffn_errors(f, x, wg, wu, wd, dy, dtype, gdt):
    """Element-wise error bounds of every result (numpy or torch, fp64).  The
    activation's slopes are at most 1.13 and its second derivative at most
    0.8, the errors of its fp32 evaluation at most 2^-19 of 1 + |g| (hardware
    exponential)."""
    u, ug = UNIT[dtype], UNIT[gdt]
    s = 2.0 ** -10 if dtype == torch.bfloat16 else E  # saved factors
    D, F, T = x.shape[1], wd.shape[1], x.shape[0]
    ab = abs
    eg, eu = 1.01 * D * E * (ab(x) @ ab(wg).T), 1.01 * D * E * (ab(x) @ ab(wu).T)
    fe = 2.0 ** -19 * (1 + ab(f["g"]))
    eb = 1.13 * eg + fe                                   # act(g)
    ea = ab(f["u"]) * (0.8 * eg + fe) + 1.2 * eu          # u·act'(g)
    eh = 1.01 * (ab(f["u"]) * eb + ab(f["b"]) * eu + eb * eu + u * ab(f["h"]))
    ea, eb = ea + 1.01 * s * ab(f["a"]) + 2.0 ** -30, eb + 1.01 * s * ab(f["b"]) + 2.0 ** -30
    edh = 1.01 * D * E * (ab(dy) @ ab(wd))
    edg = 1.01 * (ab(f["dh"]) * ea + ab(f["a"]) * edh + ea * edh + u * ab(f["dg"]))
    edu = 1.01 * (ab(f["dh"]) * eb + ab(f["b"]) * edh + eb * edh + u * ab(f["du"]))
    k = 1.01 * (2 * max(D, F, T) + 8) * E                 # the second products' own sums
    b = {"y": (eh + k * ab(f["h"])) @ ab(wd).T + u * ab(f["y"]),
         "dx": (edg + k * ab(f["dg"])) @ ab(wg) + (edu + k * ab(f["du"])) @ ab(wu) + u * ab(f["dx"]),
         "dw_gate": (edg + k * ab(f["dg"])).T @ ab(x) + ug * ab(f["dw_gate"]),
         "dw_up": (edu + k * ab(f["du"])).T @ ab(x) + ug * ab(f["dw_up"]),
         "dw_down": ab(dy).T @ (eh + k * ab(f["h"])) + ug * ab(f["dw_down"])}
    return {n: 1.02 * v + 2.0 ** -100 for n, v in b.items()}


NAMES = ("dx", "dw_gate", "dw_up", "dw_down")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ol.ACTIVATIONS)
@pytest.mark.parametrize("tokens,model,hidden", FFNS)
def test_gated_ffn(lib, tokens, model, hidden, act, dtype):
    ts = ffn_inputs(tokens, model, hidden, dtype)
    f, b = ffn_bounds(*(f64(t) for t in ts), act, dtype, dtype)
    for pad in (0, 3, 8):
        x, wg, wu, wd, dy = (strided(t, pad) for t in ts)
        y = lib.muon_gated_ffn(x, wg, wu, wd, act)
        check(y, f["y"], b["y"], ("y", pad))
        y2, saved = lib.muon_gated_ffn(x, wg, wu, wd, act, save=True)
        assert torch.equal(y, y2)
        got = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved)
        for n, g in zip(NAMES, got):
            check(g, f[n], b[n], (n, pad))
        again = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved)
        assert all(torch.equal(p, q) for p, q in zip(got, again))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [15, 16, 32, 33, 40, 47, 48, 49])
def test_gated_ffn_token_blocks(lib, tokens, dtype):
    """Tokens around whole blocks of 16, and weight gradients whose one sum
    over tokens ends inside a step of 32 (at and off a multiple of 8)."""
    ts = ffn_inputs(tokens, 300, 700, dtype)
    f, b = ffn_bounds(*(f64(t) for t in ts), "silu", dtype, dtype)
    x, wg, wu, wd, dy = (t.cuda() for t in ts)
    y, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True)
    check(y, f["y"], b["y"], "y")
    for n, g in zip(NAMES, lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved)):
        check(g, f[n], b[n], n)


@pytest.mark.parametrize("tokens,model,hidden", [(5, 24, 40), (130, 136, 264), (300, 72, 200), (64, 33, 50)])
@pytest.mark.parametrize("gdt", DTYPES)
def test_gated_ffn_grad_accumulates(lib, tokens, model, hidden, gdt):
    """Weight gradients in another type than the weights', into strided
    tensors, added to what they hold; parts of the gradient left out."""
    dtype = torch.bfloat16
    ts = ffn_inputs(tokens, model, hidden, dtype)
    f, b = ffn_bounds(*(f64(t) for t in ts), "silu", dtype, gdt)
    x, wg, wu, wd, dy = (t.cuda() for t in ts)
    _, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True)
    olds = [rand(w.shape, 40 + i, gdt) for i, w in enumerate((wg, wu, wd))]
    for pad in (0, 3, 8):
        outs = [strided(o, pad) for o in olds]
        dx, *got = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved, want_dx=False, grads=outs, accumulate=True)
        assert dx is None
        for n, g, o in zip(NAMES[1:], got, olds):
            want = f[n] + f64(o)
            check(g, want, b[n] + 1.01 * UNIT[gdt] * np.abs(want) + 2 * E * np.abs(f64(o)), (n, pad))
            if pad:
                gaps = g.as_strided((g.shape[0], pad), (g.shape[1] + pad, 1), 0)
                assert torch.isnan(gaps).all()
    only = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved, want_dweights=False)
    check(only[0], f["dx"], b["dx"], "dx alone")
    assert only[1:] == (None, None, None)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_ffn_mixed_strides(lib, dtype):
    """Every operand and result with a row stride of its own."""
    ts = ffn_inputs(70, 96, 136, dtype)
    f, b = ffn_bounds(*(f64(t) for t in ts), "silu", dtype, dtype)
    x, wg, wu, wd, dy = (strided(t, pad) for t, pad in zip(ts, (8, 16, 40, 0, 24)))
    y, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True, out=strided(ts[0], 32))
    check(y, f["y"], b["y"], "y")
    outs = [strided(t, pad) for t, pad in zip(ts[1:4], (48, 8, 56))]
    got = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved, grads=outs)
    for n, g in zip(NAMES, got):
        check(g, f[n], b[n], n)


@pytest.mark.parametrize("tokens,model,hidden", [(4096, 1024, 4096), (4096, 4096, 1024), (4001, 1032, 4104),
                                                 (2500, 4090, 1000)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_ffn_large(lib, tokens, model, hidden, dtype):
    """Sizes at which every product runs on its largest tile (each of y, dx,
    dh and the weight gradients at one of them), with ragged edges, against
    plain fp64 torch."""
    x, wg, wu, wd, dy = ffn_inputs(tokens, model, hidden, dtype)
    x, wg, wu, wd, dy = (t.cuda() for t in (x, wg, wu, wd, dy))
    X, G, U, W, Y = (t.double() for t in (x, wg, wu, wd, dy))
    f = {"g": X @ G.t(), "u": X @ U.t()}
    s = torch.sigmoid(f["g"])
    f["b"] = f["g"] * s
    f["a"] = f["u"] * (s + f["b"] * (1 - s))
    f["h"] = f["b"] * f["u"]
    f["y"] = f["h"] @ W.t()
    f["dh"] = Y @ W
    f["dg"], f["du"] = f["dh"] * f["a"], f["dh"] * f["b"]
    f["dx"] = f["dg"] @ G + f["du"] @ U
    f["dw_gate"], f["dw_up"], f["dw_down"] = f["dg"].t() @ X, f["du"].t() @ X, Y.t() @ f["h"]
    b = ffn_errors(f, X, G, U, W, Y, dtype, dtype)
    y, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True)
    got = dict(zip(("y", *NAMES), (y, *lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved))))
    for n, t in got.items():
        assert bool(((t.double() - f[n]).abs() <= b[n]).all()), n
    again = lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved)
    assert all(torch.equal(p, q) for p, q in zip(again, list(got.values())[1:]))
    # fp32 gradients added to what is there
    olds = [torch.full(w.shape, 0.5, device="cuda") for w in (wg, wu, wd)]
    lib.muon_gated_ffn_grad(dy, x, wg, wu, wd, saved, want_dx=False, grads=olds, accumulate=True)
    b32 = ffn_errors(f, X, G, U, W, Y, dtype, torch.float32)
    for n, t in zip(NAMES[1:], olds):
        assert bool(((t.double() - 0.5 - f[n]).abs() <= b32[n] + E * (0.5 + f[n].abs())).all()), n


def test_gated_ffn_empty(lib):
    x, wg, wu, wd, _ = (t.cuda() for t in ffn_inputs(4, 24, 40, torch.bfloat16))
    x = x[:0]
    y, saved = lib.muon_gated_ffn(x, wg, wu, wd, save=True)
    assert y.shape == (0, 24)
    dx, *dw = lib.muon_gated_ffn_grad(x, x, wg, wu, wd, saved)
    assert dx.shape == (0, 24) and all((g == 0).all() for g in dw)
    keep = [torch.ones_like(w) for w in (wg, wu, wd)]
    lib.muon_gated_ffn_grad(x, x, wg, wu, wd, saved, grads=keep, accumulate=True)
    assert all((g == 1).all() for g in keep)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gated_ffn_bad_rows_stay_alone(lib, dtype):
    """A token with NaN or infinity spoils its own outputs only."""
    x, wg, wu, wd, dy = (t.cuda() for t in ffn_inputs(40, 64, 96, dtype))
    y = lib.muon_gated_ffn(x, wg, wu, wd)
    x2 = x.clone()
    x2[7, 5] = float("nan")
    x2[30, 1] = float("inf")
    y2, saved = lib.muon_gated_ffn(x2, wg, wu, wd, save=True)
    rows = [i for i in range(40) if i not in (7, 30)]
    assert torch.equal(y2[rows], y[rows]) and torch.isnan(y2[7]).all()
    dx = lib.muon_gated_ffn_grad(dy, x2, wg, wu, wd, saved, want_dweights=False)[0]
    assert torch.isfinite(dx[rows]).all() and torch.isnan(dx[7]).all()


@pytest.mark.parametrize("act", ol.ACTIVATIONS)
def test_gated_ffn_large_gates(lib, act):
    """Saturated gates: no NaN from ∞·0 in the activation or its slope."""
    x = torch.tensor([[3e4], [-3e4], [3e15], [-3e15], [0.0]]).cuda()
    w = torch.ones((1, 1), device="cuda")
    y, saved = lib.muon_gated_ffn(x, w, w, w, act, save=True)
    dx = lib.muon_gated_ffn_grad(torch.ones_like(x), x, w, w, w, saved, want_dweights=False)[0]
    # y = act(v)·v: v² above, 0 below; dy/dv = 2v above, 0 below
    v = f64(x)
    ref = np.where(v > 0, v * v, 0.0)
    check(y, ref, 1e-5 * ref, "y")
    check(dx, np.where(v > 0, 2 * v, 0.0), 1e-5 * np.abs(v), "dx")


# ---------------------------------------------------- differences, autograd

def test_gradients_by_differences(lib):
    """Directional derivatives of the fp32 path by central differences: with
    step t the quotient is off by O(t²) of the third derivative and by the
    fp32 rounding of the two values over 2t (about 1e-7·|loss|/t); both are far
    below the 2% of the derivative's size allowed here."""
    emb = lib.Embedding(50, 24, scale=2.0, device="cuda")
    norm = lib.RMSNorm(24, device="cuda")
    ffn = lib.GatedFFN(24, 40, "gelu_tanh", device="cuda")
    torch.nn.init.normal_(emb.weight, std=1.0, generator=torch.Generator(device="cuda").manual_seed(1))
    ids = make_ids(64, 50, 2, torch.int64).cuda()
    target = rand((64, 24), 3, torch.float32).cuda()

    def loss():
        h = emb(ids)
        y, s = norm(h, target)
        return ((s + ffn(y)) * target).double().sum()
    out = loss()
    out.backward()
    params = [emb.weight, norm.weight, ffn.w_gate, ffn.w_up, ffn.w_down]
    for k, p in enumerate(params):
        d = rand(p.shape, 20 + k, torch.float32).cuda()
        want = float((p.grad.double() * d.double()).sum())
        scale = float(p.grad.double().norm())  # the typical size of a directional derivative
        t = 1e-2
        with torch.no_grad():
            p += t * d
            hi = float(loss())
            p -= 2 * t * d
            lo = float(loss())
            p += t * d
        assert abs((hi - lo) / (2 * t) - want) <= 0.02 * max(scale, abs(want)), (k, (hi - lo) / (2 * t), want)


def test_modules_match_functions(lib):
    """Autograd through the modules gives the functions' bits, for leading
    dimensions, broadcast and transposed incoming gradients."""
    g = torch.Generator(device="cuda").manual_seed(5)
    ffn = lib.GatedFFN(16, 24, device="cuda", dtype=torch.bfloat16)
    x = torch.randn((2, 3, 16), generator=g, device="cuda").bfloat16().requires_grad_()
    y = ffn(x)
    y.sum().backward()  # the incoming gradient is a broadcast 1
    w = (ffn.w_gate, ffn.w_up, ffn.w_down)
    ref, saved = lib.muon_gated_ffn(x.detach(), *(p.detach() for p in w), save=True)
    assert torch.equal(y, ref)
    grads = lib.muon_gated_ffn_grad(torch.ones_like(ref), x.detach(), *(p.detach() for p in w), saved)
    assert torch.equal(x.grad, grads[0]) and all(torch.equal(p.grad, q) for p, q in zip(w, grads[1:]))
    norm = lib.RMSNorm(16, device="cuda")
    a = torch.randn((16, 6), generator=g, device="cuda").t().detach().contiguous().requires_grad_()
    out = norm(a)
    c = torch.randn((16, 6), generator=g, device="cuda")
    (out.t() * c).sum().backward()
    _, _, rstd = lib.muon_rms_norm(a.detach(), norm.weight.detach())
    dx, dw = lib.muon_rms_norm_grad(c.t().contiguous(), a.detach(), norm.weight.detach(), rstd)
    assert torch.equal(a.grad, dx) and torch.equal(norm.weight.grad, dw)
    with torch.no_grad():
        assert torch.equal(ffn(x), ref)


def test_other_stream_and_graph(lib):
    """The same bits on another stream and from a replayed graph, with eager
    work between the replays."""
    ts = [t.cuda() for t in ffn_inputs(33, 64, 96, torch.bfloat16)]
    x, wg, wu, wd, dy = ts
    ids = make_ids(33, 20, 3, torch.int64).cuda()
    w = torch.ones(64, device="cuda")

    def step():
        e = lib.muon_embedding_grad(dy, ids, 20)
        n, s, r = lib.muon_rms_norm(x, w, dy)
        y, saved = lib.muon_gated_ffn(n, wg, wu, wd, save=True)
        return [e, n, s, r, y, *lib.muon_gated_ffn_grad(dy, n, wg, wu, wd, saved),
                *lib.muon_rms_norm_grad(dy, s, w, r)]
    ref = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    # an input that has to be copied to rows is copied on that stream too
    x3 = x.reshape(11, 3, 64).transpose(0, 1)
    side.wait_stream(torch.cuda.current_stream())
    y, y3 = lib.muon_gated_ffn(x, wg, wu, wd, stream=side), lib.muon_gated_ffn(x3, wg, wu, wd, stream=side)
    side.synchronize()
    assert torch.equal(y, lib.muon_gated_ffn(x, wg, wu, wd))
    assert torch.equal(y3, y.reshape(11, 3, 64).transpose(0, 1))
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


def test_example_trains(lib):
    """The example model learns: from ln(vocab) at the start (the logits of
    an untrained model say nothing about the successor) to less than half of
    it, on fresh data every step."""
    import importlib.util
    import math
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_ffn_lm.py")
    spec = importlib.util.spec_from_file_location("train_ffn_lm", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.train(steps=60, tokens=2048, vocab=256, model=128, hidden=384, depth=2, log=lambda s: None)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.5 * math.log(256)
