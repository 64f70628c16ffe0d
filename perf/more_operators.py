"""Cases that measure the attention half of a training block: the rotation of
queries and keys by their positions and its gradient, differential attention
(the difference of two softmax maps), forward and forward + backward, and
dropout with the residual's addition and its gradient.

Each case names its operator, its direction and its sizes.  ``run`` computes a
pass either in plain torch operations (fp32 throughout, angles in fp64, rounded
once at the end) or, where ``own`` is true, through the package's public entry
points.  ``exact`` computes the same results from the definitions in fp64.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------- the cases
#
# Attention: `heads` output heads, each the difference of two maps, so q has
# 2·heads heads of `dim` values, k 2·kv heads, v kv heads of 2·dim values.
# 28 and 4 heads of 64 make the q, k and v matrices of the benchmark's layer
# (3584×3584, 512×3584, 512×3584).  `seqs` > 0: that many sequences of
# different lengths packed one after another (`cut` fixes where), the last of
# `tokens` rows behind them unused.

def listed():
    return [
        # one token of a decoding loop: latency alone
        dict(name="rotary decode", op="rotary", batch=1, tokens=1, heads=56, kv=8, dim=64, rot=64, dtype="bf16",
             inter=False, far=True),
        # a training batch
        dict(name="rotary batch", op="rotary", batch=4, tokens=4096, heads=56, kv=8, dim=64, rot=64, dtype="bf16",
             inter=False, far=False),
        # a small fp32 model that rotates part of each head, odd sizes, far positions
        dict(name="rotary grad odd", op="rotary_grad", batch=3, tokens=1001, heads=6, kv=2, dim=72, rot=38, dtype="f32",
             inter=True, far=True),
        # a small fp32 model's batch with an odd width
        dict(name="dropout odd", op="dropout", tokens=1003, model=1021, dtype="f32", residual=True, p=0.1),
        # a training batch's block output on its way into the residual stream
        dict(name="dropout batch", op="dropout", tokens=16384, model=3584, dtype="bf16", residual=True, p=0.1),
        # its gradient
        dict(name="dropout grad batch", op="dropout_grad", tokens=16384, model=3584, dtype="bf16", p=0.1),
        # one decoded token against a long context: keys and values are read once
        dict(name="attention decode", op="attention", batch=1, queries=1, tokens=16384, heads=28, kv=4, dim=64,
             dtype="bf16", causal=True, seqs=0),
        # a prompt's forward pass
        dict(name="attention prompt", op="attention", batch=1, queries=4096, tokens=4096, heads=28, kv=4, dim=64,
             dtype="bf16", causal=True, seqs=0),
        # a small fp32 model's step, odd sizes: forward, then all gradients
        dict(name="attention train odd", op="attention_train", batch=2, queries=333, tokens=333, heads=6, kv=2, dim=40,
             dtype="f32", causal=True, seqs=0),
        # documents of different lengths packed into one row: forward, then all gradients
        dict(name="attention train packed", op="attention_train", batch=1, queries=8192, tokens=8192, heads=28, kv=4,
             dim=64, dtype="bf16", causal=True, seqs=11, cut=5),
        # wide heads: forward, then all gradients
        dict(name="attention train wide", op="attention_train", batch=1, queries=2048, tokens=2048, heads=14, kv=2,
             dim=128, dtype="bf16", causal=True, seqs=0),
        # a training batch: forward, then all gradients
        dict(name="attention train batch", op="attention_train", batch=4, queries=4096, tokens=4096, heads=28, kv=4,
             dim=64, dtype="bf16", causal=True, seqs=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width over the whole range: often a multiple of 128, sometimes of 8,
    sometimes any number."""
    n = _log_int(rng, lo, hi)
    step = rng.choice((128, 128, 8, 1))
    return max(step, min(hi, n // step * step)) if step > 1 else n


_LARGEST = 4 * 28 * 64 * 4096 ** 2  # of "attention train batch": batch · heads · dim · tokens²


def draw(rng):
    op = rng.choice(("rotary", "rotary_grad", "dropout", "dropout_grad", "attention", "attention", "attention_train",
                     "attention_train", "attention_train"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("dropout", "dropout_grad"):
        case = dict(op=op, tokens=_log_int(rng, 1, 16384), model=_width(rng, 64, 3584), dtype=dtype,
                    p=rng.choice((0.05, 0.1, 0.3)))
        return dict(case, residual=rng.random() < 0.7) if op == "dropout" else case
    kv = rng.choice((1, 2, 4))
    group = rng.choice((1, 2, 3, 7))
    if op in ("rotary", "rotary_grad"):
        dim = rng.choice((64, 64, 128, 80, 72, 36))
        rot = rng.choice((dim, dim, dim // 2, dim // 4 * 2))
        return dict(op=op, batch=rng.randint(1, 4), tokens=_log_int(rng, 1, 4096), heads=2 * kv * group, kv=2 * kv,
                    dim=dim, rot=rot, dtype=dtype, inter=rng.random() < 0.5, far=rng.random() < 0.5)
    dim = rng.choice((64, 64, 64, 128, 32, 40, 80))
    case = dict(op=op, batch=rng.randint(1, 4), heads=kv * group, kv=kv, dim=dim, dtype=dtype,
                causal=rng.random() < 0.8)
    # fp32 products run an order of magnitude slower than half-precision ones
    tokens = _log_int(rng, 1, 4096 if dtype == "bf16" else 1024)
    kind = rng.choice(("same", "same", "packed", "few"))
    if op == "attention_train" or kind != "few":  # the widest heads without a mask: fewer tokens
        while case["batch"] * case["heads"] * case["dim"] * tokens ** 2 * (1 if case["causal"] else 2) > _LARGEST:
            tokens //= 2
    if kind == "packed" and tokens >= 16:
        return dict(case, batch=1, queries=tokens, tokens=tokens, seqs=rng.randint(1, 12), cut=rng.randint(0, 10 ** 6))
    if kind == "few" and op == "attention":  # a few tokens against a cache
        return dict(case, queries=rng.randint(1, min(8, tokens)), tokens=tokens, seqs=0)
    return dict(case, queries=tokens, tokens=tokens, seqs=0)


def _lengths(case):
    """Lengths of the packed sequences: one empty where there are several, and
    a few rows left behind the last."""
    rng = random.Random(case["cut"])
    used, n = case["tokens"] - case["tokens"] // 100, case["seqs"]
    cuts = sorted(rng.randint(1, used) for _ in range(n - 1))
    ends = cuts + [used]
    lengths = [b - a for a, b in zip([0] + cuts, ends)]
    if n > 3:  # an empty document
        lengths[2] += lengths[1]
        lengths[1] = 0
    return lengths


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dt)

    op, s = case["op"], {"case": case}
    if op in ("dropout", "dropout_grad"):
        shape = (case["tokens"], case["model"])
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ int(seed), 3 + int(seed)
        s["x"] = normal(*shape, std=1.0 if op == "dropout" else 1e-2)
        if op == "dropout" and case["residual"]:
            s["residual"] = normal(*shape, std=4.0)
        return s
    if op in ("rotary", "rotary_grad"):
        b, t, d, r = case["batch"], case["tokens"], case["dim"], case["rot"]
        s["q"], s["k"] = normal(b, t, case["heads"], d), normal(b, t, case["kv"], d)
        s["freqs"] = 1e6 ** (-torch.arange(r // 2, dtype=torch.float64, device=dev) * 2 / r)
        if case["far"]:  # positions of a long context, another stretch in each row
            s["positions"] = torch.randint(0, 10 ** 6, (b, 1), generator=gen, device=dev) + torch.arange(t, device=dev)
        return s
    b, tq, tk, h, kv, d = (case[n] for n in ("batch", "queries", "tokens", "heads", "kv", "dim"))
    packed = case["seqs"] > 0
    lead = (tq,) if packed else (b, tq)
    leadk = (tk,) if packed else (b, tk)
    # rows whose maps are flat and rows whose maps are sharp
    sharp = torch.exp(0.5 * torch.randn((*lead, 1, 1), generator=gen, device=dev))
    s["q"] = (torch.randn((*lead, 2 * h, d), generator=gen, device=dev) * sharp).to(dt)
    s["k"] = normal(*leadk, 2 * kv, d)
    s["v"] = normal(*leadk, kv, 2 * d)
    s["lam"] = 0.2 + 0.6 * torch.rand(h, generator=gen, device=dev)
    if packed:
        lengths = _lengths(case)
        ends = torch.tensor([0] + lengths).cumsum(0)
        s["spans"] = [(int(a), int(z)) for a, z in zip(ends[:-1], ends[1:])]
        s["offsets"] = ends.to(device=dev, dtype=torch.int32)
    if op == "attention_train":
        s["dout"] = normal(*lead, h, 2 * d, std=1e-2)
    return s


# ------------------------------------------------------------------ one pass

_LOW = 0xFFFFFFFF


def _keep(shape, p, seed, offset, dev):
    """The words of Philox4x32-10, counter (index / 4, offset), key seed, word
    index % 4, that are at least p·2^32."""
    n = math.prod(shape)
    i = torch.arange((n + 3) // 4, dtype=torch.int64, device=dev)
    c = [i & _LOW, i >> 32, torch.full_like(i, offset & _LOW), torch.full_like(i, (offset >> 32) & _LOW)]
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # 64-bit products, their bits kept when they wrap
        c = [((b >> 32) & _LOW) ^ c[1] ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c[3] ^ k1, a & _LOW]
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    words = torch.stack(c, dim=1).reshape(-1)[:n]
    return (words >= round(p * 2 ** 32)).reshape(shape)


def _rotate(x, cos, sin, rot, inter):
    f = x.float()
    y = f.clone()
    if inter:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = f[..., :rot // 2], f[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, a * sin + b * cos
    return y.to(x.dtype)


def _maps(q, k, causal):
    """Both softmax maps of one sequence, each heads × queries × keys."""
    (tq, h2, d), (tk, kv2, _) = q.shape, k.shape
    group = h2 // kv2
    hidden = None
    if causal:
        i, j = torch.arange(tq, device=q.device)[:, None], torch.arange(tk, device=q.device)[None, :]
        hidden = j > i + (tk - tq)
    out = []
    for m in (0, 1):
        qm = q[:, m::2].transpose(0, 1)  # heads × queries × dim
        km = k[:, m::2].transpose(0, 1).repeat_interleave(group, dim=0)
        s = (qm @ km.transpose(1, 2)).mul_(1.0 / math.sqrt(d))
        if hidden is not None:
            s.masked_fill_(hidden, float("-inf"))
        s = s.sub_(s.amax(dim=2, keepdim=True).clamp_(min=-3e38)).exp_()
        out.append(s.div_(s.sum(dim=2, keepdim=True).clamp_(min=1e-38)))
    return out


def _attend(q, k, v, lam, causal, dout=None):
    """One sequence: its output, and with dout its gradients."""
    q, k, v = q.float(), k.float(), v.float()
    (tq, h2, d), (tk, kv, dv) = q.shape, v.shape
    h, group = h2 // 2, h2 // 2 // kv
    if tq == 0 or tk == 0:
        zero = [torch.zeros((tq, h, dv), device=q.device)]
        return zero if dout is None else zero + [torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v),
                                                 torch.zeros_like(lam)]
    p1, p2 = _maps(q, k, causal)
    vh = v.transpose(0, 1).repeat_interleave(group, dim=0)
    a = p1 - lam[:, None, None] * p2
    out = [(a @ vh).transpose(0, 1)]
    if dout is None:
        return out
    do = dout.float().transpose(0, 1)
    dv_ = (a.transpose(1, 2) @ do).reshape(kv, group, tk, dv).sum(dim=1).transpose(0, 1)
    da = do @ vh.transpose(1, 2)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    sums = [(p * da).sum(dim=2, keepdim=True) for p in (p1, p2)]
    for m, p in enumerate((p1, p2)):
        ds = p * (da - sums[m]) * (1.0 / math.sqrt(d))
        if m:
            ds = ds * -lam[:, None, None]
        km = k[:, m::2].transpose(0, 1).repeat_interleave(group, dim=0)
        dq[:, m::2] = (ds @ km).transpose(0, 1)
        dkm = ds.transpose(1, 2) @ q[:, m::2].transpose(0, 1)
        dk[:, m::2] = dkm.reshape(kv, group, tk, d).sum(dim=1).transpose(0, 1)
    return out + [dq, dk, dv_, -sums[1].sum(dim=(1, 2))]


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _DTYPES[case["dtype"]]
    if op in ("dropout", "dropout_grad"):
        y = s["x"].float() * (1.0 / (1.0 - case["p"]))
        y = torch.where(_keep(y.shape, case["p"], s["seed"], s["offset"], y.device), y, torch.zeros_like(y))
        if "residual" in s:
            y = y + s["residual"].float()
        return y.to(dt)
    if op in ("rotary", "rotary_grad"):
        q, k = s["q"], s["k"]
        pos = s["positions"] if "positions" in s else torch.arange(case["tokens"], device=q.device)[None, :]
        angle = pos.double()[:, :, None, None] * s["freqs"]
        cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
        if op == "rotary_grad":  # the transposed rotation
            sin = -sin
        return {n: _rotate(t, cos, sin, case["rot"], case["inter"]) for n, t in (("q", q), ("k", k))}
    q, k, v, lam, causal, dout = s["q"], s["k"], s["v"], s["lam"], case["causal"], s.get("dout")
    names = ("out", "dq", "dk", "dv", "dlam")
    if case["seqs"]:
        like = {"out": (*q.shape[:1], case["heads"], 2 * case["dim"]), "dq": q.shape, "dk": k.shape, "dv": v.shape}
        res = {n: torch.zeros(sh, dtype=dt, device=q.device) for n, sh in like.items() if n == "out" or dout is not None}
        if dout is not None:
            res["dlam"] = torch.zeros_like(lam)
        for a, z in s["spans"]:
            got = _attend(q[a:z], k[a:z], v[a:z], lam, causal, dout[a:z] if dout is not None else None)
            for n, t in zip(names, got):
                if n == "dlam":
                    res[n] += t
                else:
                    res[n][a:z] = t.to(dt)
    else:
        each = [_attend(q[b], k[b], v[b], lam, causal, dout[b] if dout is not None else None)
                for b in range(case["batch"])]
        res = {n: torch.stack(t) for n, t in zip(names, zip(*each))}
        res = {n: t.sum(dim=0) if n == "dlam" else t.to(dt) for n, t in res.items()}
    return res["out"] if dout is None else res


def _own(s):
    import muon_newton_schulz_06_amd as mns
    case = s["case"]
    op = case["op"]
    if op == "dropout":
        return mns.muon_dropout(s["x"], case["p"], s["seed"], s["offset"], residual=s.get("residual"))
    if op == "dropout_grad":
        return mns.muon_dropout_grad(s["x"], case["p"], s["seed"], s["offset"])
    if op in ("rotary", "rotary_grad"):
        call = mns.muon_rotary if op == "rotary" else mns.muon_rotary_grad
        q, k = call(s["q"], s["k"], s["freqs"], positions=s.get("positions"), interleaved=case["inter"])
        return {"q": q, "k": k}
    qkv = (s["q"], s["k"], s["v"], s["lam"])
    how = dict(causal=case["causal"], offsets=s.get("offsets"))
    if op == "attention":
        return mns.muon_diff_attention(*qkv, **how)
    out, saved = mns.muon_diff_attention(*qkv, **how, save=True)
    dq, dk, dv, dlam = mns.muon_diff_attention_grad(s["dout"], *qkv, out, saved, **how)
    return {"out": out, "dq": dq, "dk": dk, "dv": dv, "dlam": dlam}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- 64-bit results

def _mul32(a, m):
    """(high, low) 32 bits of a·m from 16-bit halves."""
    a0, a1, m0, m1 = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = a0 * m1 + ((a0 * m0) >> 16)
    cross = a1 * m0 + (mid & 0xFFFF)
    return a1 * m1 + (mid >> 16) + (cross >> 16), ((cross & 0xFFFF) << 16) | ((a0 * m0) & 0xFFFF)


def _exact_head(q1, q2, k1, k2, v, lam, causal):
    def soft(a, b):
        z = (a @ b.t()) / math.sqrt(a.shape[1])
        if causal:
            z = z + torch.full_like(z, float("-inf")).triu(b.shape[0] - a.shape[0] + 1)
        return torch.softmax(z, dim=1)
    return soft(q1, k1) @ v - lam * (soft(q2, k2) @ v)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("dropout", "dropout_grad"):
        x = s["x"].double()
        n = x.numel()
        at = torch.arange(n, dtype=torch.int64, device=x.device)
        word = torch.empty(n, dtype=torch.int64, device=x.device)
        for part in range(0, n, 1 << 24):
            i = at[part:part + (1 << 24)]
            c0, c1 = (i >> 2) & _LOW, i >> 34
            c2, c3 = torch.full_like(i, s["offset"] & _LOW), torch.full_like(i, s["offset"] >> 32)
            for r in range(10):
                h0, l0 = _mul32(c0, 0xD2511F53)
                h1, l1 = _mul32(c2, 0xCD9E8D57)
                key = [((s["seed"] & _LOW) + r * 0x9E3779B9) & _LOW, ((s["seed"] >> 32) + r * 0xBB67AE85) & _LOW]
                c0, c1, c2, c3 = h1 ^ c1 ^ key[0], l1, h0 ^ c3 ^ key[1], l0
            w = i & 3
            word[part:part + (1 << 24)] = torch.where(w < 2, torch.where(w == 0, c0, c1), torch.where(w == 2, c2, c3))
        y = x / (1.0 - case["p"])
        y[(word < round(case["p"] * 2 ** 32)).reshape(x.shape)] = 0.0
        return y + s["residual"].double() if "residual" in s else y
    if op in ("rotary", "rotary_grad"):
        pos = s["positions"] if "positions" in s else torch.arange(case["tokens"], device=s["q"].device)[None, :]
        turn = pos.double()[..., None, None] * s["freqs"]
        turn = torch.polar(torch.ones_like(turn), -turn if op == "rotary_grad" else turn)
        rot, out = case["rot"], {}
        for n in ("q", "k"):
            x = s[n].double()
            if case["inter"]:
                z = torch.view_as_complex(x[..., :rot].unflatten(-1, (-1, 2)).contiguous())
                y = torch.view_as_real(z * turn).flatten(-2)
            else:
                z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
                y = torch.cat((z.real, z.imag), dim=-1)
            out[n] = torch.cat((y, x[..., rot:]), dim=-1)
        return out
    train = op == "attention_train"
    one = case["seqs"] > 0
    q, k, v = (s[n].double()[None] if one else s[n].double() for n in ("q", "k", "v"))
    lam = s["lam"].double()
    res = {"out": torch.zeros((*q.shape[:2], case["heads"], 2 * case["dim"]), dtype=torch.float64, device=q.device)}
    if train:
        dout = s["dout"].double()[None] if one else s["dout"].double()
        res.update(dq=torch.zeros_like(q), dk=torch.zeros_like(k), dv=torch.zeros_like(v), dlam=torch.zeros_like(lam))
    group = case["heads"] // case["kv"]
    for b in range(q.shape[0]):
        for a, z in s.get("spans", [(0, case["tokens"])]):
            if z == a:
                continue
            rows = slice(a, z) if one else slice(None)
            for h in range(case["heads"]):
                g = h // group
                args = [q[b, rows, 2 * h], q[b, rows, 2 * h + 1], k[b, a:z, 2 * g], k[b, a:z, 2 * g + 1], v[b, a:z, g], lam[h]]
                if not train:
                    res["out"][b, rows, h] = _exact_head(*args, case["causal"])
                    continue
                args = [t.detach().clone().requires_grad_() for t in args]
                o = _exact_head(*args, case["causal"])
                res["out"][b, rows, h] = o.detach()
                d = torch.autograd.grad(o, args, dout[b, rows, h])
                res["dq"][b, rows, 2 * h], res["dq"][b, rows, 2 * h + 1] = d[0], d[1]
                res["dk"][b, a:z, 2 * g] += d[2]
                res["dk"][b, a:z, 2 * g + 1] += d[3]
                res["dv"][b, a:z, g] += d[4]
                res["dlam"][h] += d[5]
    if one:
        res = {n: t if n == "dlam" else t[0] for n, t in res.items()}
    return res if train else res["out"]


# --------------------------------------------------- what a pass cannot avoid

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op = case["op"]
    if op in ("dropout", "dropout_grad"):
        n = case["tokens"] * case["model"]
        return {"bytes": (3 if case.get("residual") else 2) * n * e, "flops": 2 * n}
    if op in ("rotary", "rotary_grad"):
        rows = case["batch"] * case["tokens"]
        heads = case["heads"] + case["kv"]
        return {"bytes": 2 * rows * heads * case["dim"] * e + 8 * rows * case["far"] + 4 * case["rot"],
                "flops": 3 * rows * heads * case["rot"]}
    b, tq, tk, h, kv, d = (case[n] for n in ("batch", "queries", "tokens", "heads", "kv", "dim"))
    spans = [(n, n) for n in _lengths(case)] if case["seqs"] else [(tq, tk)] * b
    # causal: row i of tq meets tk - tq + i + 1 keys
    pairs = sum(q * k - (q * (q - 1) // 2 if case["causal"] else 0) for q, k in spans)
    q, k, v, out = b * tq * 2 * h * d, b * tk * 2 * kv * d, b * tk * kv * 2 * d, b * tq * h * 2 * d
    # per pair and head two scores and one weighted sum of values: 8·d; the
    # gradients: the scores again, dA, dV, and dK and dQ of both maps: 20·d
    if op == "attention":
        return {"bytes": (q + k + v + out) * e, "flops": 8.0 * d * h * pairs}
    return {"bytes": (3 * q + 3 * k + 3 * v + 4 * out) * e, "flops": 28.0 * d * h * pairs}
