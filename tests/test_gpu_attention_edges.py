"""Attention calls at the edges of what the header allows."""
import pytest
import torch

from test_gpu_attention import DTYPES, attention_inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 72, 128])
@pytest.mark.parametrize("batch,queries,keys", [(1, 0, 300), (2, 0, 4096), (0, 5, 300), (0, 5, 4096), (0, 0, 1000)])
def test_no_queries_or_no_batch(lib, batch, queries, keys, dim, dtype):
    """Against many keys too: no results, and gradients of zero for all of them."""
    q, k, v, lam, do = (t.cuda() for t in attention_inputs(batch, queries, keys, 4, 2, dim, dtype))
    sizes = (batch, queries, keys, 4, 2, dim, dtype)
    assert lib.diff_attention_saved_size(*sizes) == 0
    ws = torch.full((max(lib.diff_attention_workspace_size(*sizes, grad=True), 256),), 255, dtype=torch.uint8, device="cuda")
    for causal in (True, False):
        out, saved = lib.muon_diff_attention(q, k, v, lam, causal=causal, save=True)
        assert out.shape == do.shape and saved.numel() == 0
        for kw in (dict(), dict(workspace=ws)):
            grads = lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved, causal=causal, **kw)
            assert [g.shape for g in grads] == [q.shape, k.shape, v.shape, lam.shape] and not any(g.any() for g in grads)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("queries,keys,heads,kv", [(40, 33, 4, 2), (300, 200, 3, 1), (100, 60, 7, 1), (5, 2, 4, 4), (70, 3, 6, 2),
                                                   (333, 1, 2, 1), (520, 300, 2, 2)])
def test_rows_that_see_no_key(lib, queries, keys, heads, kv, dim, dtype):
    """More queries than keys, causal: the first rows see nothing.  Whatever is in
    their q and dout reaches no gradient."""
    blind = queries - keys
    q, k, v, lam, do = (t.cuda() for t in attention_inputs(2, queries, keys, heads, kv, dim, dtype))
    q[:, :blind], do[:, :blind] = 0, 0
    ref, saved = lib.muon_diff_attention(q, k, v, lam, save=True)
    refs = lib.muon_diff_attention_grad(do, q, k, v, lam, ref, saved)
    assert not ref[:, :blind].any() and not refs[0][:, :blind].any() and all(torch.isfinite(g).all() for g in refs)
    for bad_q, bad_do in ((float("nan"), float("nan")), (float("inf"), 1.0), (1.0, float("-inf")), (float("-inf"), float("nan"))):
        q[:, :blind], do[:, :blind] = bad_q, bad_do
        out, saved = lib.muon_diff_attention(q, k, v, lam, save=True)
        grads = lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved)
        assert torch.equal(out, ref)
        for name, a, b in zip(("dq", "dk", "dv", "dlam"), grads, refs):
            assert torch.equal(a, b), (name, bad_q, bad_do)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("queries,keys,heads,kv", [(40, 33, 4, 2), (300, 200, 3, 1), (5, 2, 4, 4), (333, 1, 2, 1), (3000, 2990, 1, 1)])
def test_results_of_rows_that_see_no_key(lib, queries, keys, heads, kv, dim, dtype):
    """They are zeros whatever the values hold, by one pass and by splits of the keys."""
    blind = queries - keys
    q, k, v, lam, do = (t.cuda() for t in attention_inputs(2, queries, keys, heads, kv, dim, dtype))
    ref = lib.muon_diff_attention(q, k, v, lam)
    for bad in (float("nan"), float("inf")):
        v[:, 0, :, 3] = bad
        out, saved = lib.muon_diff_attention(q, k, v, lam, save=True)
        assert not out[:, :blind].any() and torch.equal(lib.muon_diff_attention(q, k, v, lam)[:, :blind], out[:, :blind])
        assert not torch.isfinite(out[:, blind:, :, 3]).any() and torch.equal(out[:, blind:, :, 4:], ref[:, blind:, :, 4:])
        assert not lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved)[0][:, :blind].any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("tokens", [20, 150])
def test_bad_keys_show_in_the_gradients(lib, tokens, bad, dim, dtype):
    """A key that makes a row's sum NaN leaves no finite gradient where that row
    has a part, and changes nothing elsewhere."""
    q, k, v, lam, do = (t.cuda() for t in attention_inputs(2, tokens, tokens, 4, 2, dim, dtype))
    out, saved = lib.muon_diff_attention(q, k, v, lam, causal=False, save=True)
    refs = lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved, causal=False)
    k[1, 7, 2] = bad  # first map of the second key head
    out, saved = lib.muon_diff_attention(q, k, v, lam, causal=False, save=True)
    dq, dk, dv, dlam = lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved, causal=False)
    assert not torch.isfinite(out[1, :, 2:]).any()
    # (the second map's row sums stand apart from the first's: its gradients stay)
    assert not torch.isfinite(dv[1, :, 1]).any()
    assert not torch.isfinite(dk[1, :, 2]).any() and not torch.isfinite(dq[1, :, 4::2]).any()
    for got, ref, heads in ((dq, refs[0], 4), (dk, refs[1], 2), (dv, refs[2], 1)):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1, :, :heads], ref[1, :, :heads])
    assert torch.equal(dlam[:2], refs[3][:2])


# Tokens, and one of them that is bad: in the first, a middle and the last row of
# tiles and blocks, with groups that put several heads' rows into one tile.
HIDDEN = [(40, 20, 4, 2), (40, 0, 2, 2), (200, 199, 3, 1), (333, 150, 7, 1), (520, 300, 2, 2), (130, 31, 4, 4), (20, 9, 2, 1)]
BAD = [float("nan"), float("inf"), float("-inf")]


def clean(lib, tokens, heads, kv, dim, dtype, packed):
    """(tensors, what calls take beside them, results and gradients)"""
    ts = [t.cuda() for t in attention_inputs(1 if packed else 2, tokens, tokens, heads, kv, dim, dtype)]
    kw = {}
    if packed:  # the bad token's sequence begins at 0
        ts = [t[0] if t.dim() == 4 else t for t in ts]
        kw = dict(offsets=torch.tensor([0, tokens], dtype=torch.int32, device="cuda"))
    return ts, kw, passes(lib, ts, kw)


def passes(lib, ts, kw):
    q, k, v, lam, do = ts
    out, saved = lib.muon_diff_attention(q, k, v, lam, save=True, **kw)
    assert torch.equal(out.nan_to_num(7.0), lib.muon_diff_attention(q, k, v, lam, **kw).nan_to_num(7.0))
    return out, *lib.muon_diff_attention_grad(do, q, k, v, lam, out, saved, **kw)


def same_but(got, ref, hit, what):
    """Bits outside `hit` (True where the bad value has a part)."""
    assert torch.equal(got[~hit], ref[~hit]), what


def all_bad(got, hit, what):
    assert not torch.isfinite(got[hit]).any(), what


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("tokens,at,heads,kv", HIDDEN)
def test_hidden_values(lib, tokens, at, heads, kv, packed, dim, dtype):
    """An infinity or NaN in a value of token `at` reaches the same value of the
    results from that token on, and nothing else of them."""
    ts, kw, ref = clean(lib, tokens, heads, kv, dim, dtype, packed)
    g = heads // kv
    for bad in BAD:
        v = ts[2].clone()
        v[..., at, kv - 1, 5] = bad
        got = passes(lib, [*ts[:2], v, *ts[3:]], kw)
        hit = torch.zeros_like(ref[0], dtype=torch.bool)
        hit[..., at:, heads - g:, 5] = True
        same_but(got[0], ref[0], hit, ("out", bad))
        all_bad(got[0], hit, ("out", bad))
        hit = torch.zeros_like(ref[1], dtype=torch.bool)
        hit[..., at:, 2 * (heads - g):, :] = True
        same_but(got[1], ref[1], hit, ("dq", bad))
        assert torch.equal(got[3], ref[3])  # the values have no part in their gradient


def bad_rows(lib, tokens, at, heads, kv, dim, dtype, packed, which):
    """A bad value of token `at` in a query or the incoming gradient reaches the
    gradients of that row and of the keys that it sees, and nothing else."""
    ts, kw, ref = clean(lib, tokens, heads, kv, dim, dtype, packed)
    g, h = heads // kv, heads - 1
    for bad in BAD:
        new = [t.clone() for t in ts]
        if which == "q":
            new[0][..., at, 2 * h:2 * h + 2, :] = bad
        else:
            new[4][..., at, h, 3] = bad
        out, dq, dk, dv, dlam = passes(lib, new, kw)
        hit = [torch.zeros_like(t, dtype=torch.bool) for t in ref]
        hit[0][..., at, h, :] = which == "q"
        hit[1][..., at, 2 * h:2 * h + 2, :] = True
        hit[2][..., :at + 1, 2 * (kv - 1):, :] = True
        hit[3][..., :at + 1, kv - 1, :] = True
        hit[4][h] = True
        for name, a, b, m in zip(("out", "dq", "dk", "dv", "dlam"), (out, dq, dk, dv, dlam), ref, hit):
            same_but(a, b, m, (name, bad))
        # (the row that sees one key has no gradient of its scores)
        if at:
            all_bad(dq, hit[1], ("dq", bad))
            all_bad(dk, hit[2], ("dk", bad))
        if which == "q":
            all_bad(dv, hit[3], ("dv", bad))
        else:  # the same value of the values alone
            all_bad(dv[..., :at + 1, kv - 1, 3], ..., ("dv", bad))
            hit[3][..., [i for i in range(2 * dim) if i != 3]] = False
            same_but(dv, ref[3], hit[3], ("dv", bad))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("which", ["q", "dout"])
@pytest.mark.parametrize("tokens,at,heads,kv", HIDDEN)
def test_hidden_rows(lib, tokens, at, heads, kv, which, packed, dim, dtype):
    bad_rows(lib, tokens, at, heads, kv, dim, dtype, packed, which)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("tokens,at,heads,kv", HIDDEN)
def test_hidden_keys(lib, tokens, at, heads, kv, packed, dim, dtype):
    """A key without finite values reaches no row before it."""
    ts, kw, ref = clean(lib, tokens, heads, kv, dim, dtype, packed)
    g = heads // kv
    for bad in BAD:
        k = ts[1].clone()
        k[..., at, 2 * (kv - 1), :] = bad  # the first map's
        out, dq, dk, dv, dlam = passes(lib, [ts[0], k, *ts[2:]], kw)
        hit = torch.zeros_like(out, dtype=torch.bool)
        hit[..., at:, heads - g:, :] = True
        same_but(out, ref[0], hit, ("out", bad))
        all_bad(out, hit, ("out", bad))
        hit = torch.zeros_like(dq, dtype=torch.bool)
        hit[..., at:, 2 * (heads - g)::2, :] = True
        same_but(dq, ref[1], hit, ("dq", bad))
        if at:
            all_bad(dq, hit, ("dq", bad))
        assert torch.equal(dk[..., :2 * (kv - 1), :], ref[2][..., :2 * (kv - 1), :])
        assert torch.equal(dk[..., 2 * kv - 1, :], ref[2][..., 2 * kv - 1, :])  # the second map's
        assert torch.equal(dlam, ref[4])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128, 40])
@pytest.mark.parametrize("queries,keys,heads,kv", [(8, 4096, 4, 2), (5, 700, 6, 2), (40, 5000, 3, 1), (3, 1, 2, 2), (300, 5000, 2, 1)])
def test_hidden_among_many_keys(lib, queries, keys, heads, kv, dim, dtype):
    """The last rows of a long context, its keys split: a bad key or value that only
    some of them see, and one that all see."""
    ts = [t.cuda() for t in attention_inputs(2, queries, keys, heads, kv, dim, dtype)]
    ref = passes(lib, ts, {})
    g = heads // kv
    for at in {max(keys - 1 - queries // 3, 0), keys - 1, max(keys - queries, 0), keys // 2}:
        first = max(at - (keys - queries), 0)  # the first row that sees it
        for bad in BAD:
            for which, head, part in ((1, 2 * (kv - 1), slice(None)), (2, kv - 1, 5)):
                new = [t.clone() for t in ts]
                new[which][:, at, head, part] = bad
                out, dq, dk, dv, dlam = passes(lib, new, {})
                hit = torch.zeros_like(out, dtype=torch.bool)
                hit[:, first:, heads - g:, part] = True
                same_but(out, ref[0], hit, ("out", at, bad))
                all_bad(out, hit, ("out", at, bad))
                hit = torch.zeros_like(dq, dtype=torch.bool)
                hit[:, first:, 2 * (heads - g):: 2 if which == 1 else 1] = True
                same_but(dq, ref[1], hit, ("dq", at, bad))
                if which == 2:
                    assert torch.equal(dv, ref[3])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_bad_sequences_stay_alone(lib, causal, dim, dtype):
    """Nothing of a packed batch's sequence reaches its neighbours."""
    tokens, at = 300, (97, 161)
    q, k, v, lam, do = (t.cuda() if t.dim() == 1 else t[0].cuda() for t in attention_inputs(1, tokens, tokens, 3, 1, dim, dtype))
    off = torch.tensor([0, *at, tokens], dtype=torch.int32, device="cuda")
    kw = dict(offsets=off, causal=causal)
    ref = passes(lib, [q, k, v, lam, do], kw)
    for bad in BAD:
        new = [t.clone() for t in (q, k, v, lam, do)]
        for i in (0, 1, 2, 4):
            new[i][at[0]:at[1]] = bad
        got = passes(lib, new, kw)
        for name, a, b in zip(("out", "dq", "dk", "dv"), got, ref):
            assert torch.equal(a[:at[0]], b[:at[0]]) and torch.equal(a[at[1]:], b[at[1]:]), (name, bad)
            assert name == "dq" or not torch.isfinite(a[at[0] + 1:at[1]]).any(), (name, bad)
