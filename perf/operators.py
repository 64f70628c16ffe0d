"""Cases that measure the training-block operators: the embedding lookup and
its gradient, the RMS norm with the residual's addition and its gradient, and
the gated feed-forward block, forward and forward + backward.

Each case names its operator, its direction and its sizes.  ``run`` computes a
pass either in plain torch operations (fp32 throughout, rounded once at the
end) or, where ``own`` is true, through the package's public entry points.
``exact`` computes the same results from the definitions in fp64.
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6
_ACTS = ("silu", "gelu", "gelu_tanh")


# ----------------------------------------------------------------- the cases

def listed():
    return [
        # one token of a decoding loop: latency alone
        dict(name="embed decode", op="embed", tokens=1, vocab=32000, model=512, dtype="bf16", pad=0.0),
        # a training batch's lookup at the width of the benchmark's matrices
        dict(name="embed batch", op="embed", tokens=16384, vocab=131072, model=3584, dtype="bf16", pad=0.0),
        # a small fp32 model with an odd vocabulary and width, padded batches
        dict(name="embed grad odd", op="embed_grad", tokens=4093, vocab=50001, model=1023, dtype="f32", pad=0.03),
        # the gradient of a whole training batch, tokens distributed as words are
        dict(name="embed grad batch", op="embed_grad", tokens=16384, vocab=131072, model=3584, dtype="bf16", pad=0.0),
        # one decoded token
        dict(name="norm decode", op="norm", tokens=1, model=3584, dtype="bf16", residual=True),
        # a training batch
        dict(name="norm batch", op="norm", tokens=16384, model=3584, dtype="bf16", residual=True),
        # an fp32 model with odd sizes
        dict(name="norm grad odd", op="norm_grad", tokens=1000, model=1001, dtype="f32", residual=False),
        # a training batch's backward pass
        dict(name="norm grad batch", op="norm_grad", tokens=16384, model=3584, dtype="bf16", residual=True),
        # one decoded token through the benchmark's FFN: every weight is read once
        dict(name="ffn decode", op="ffn", tokens=1, model=3584, hidden=18944, dtype="bf16", act="silu"),
        # a prompt's forward pass
        dict(name="ffn prompt", op="ffn", tokens=2048, model=3584, hidden=18944, dtype="bf16", act="silu"),
        # a small fp32 model's step, odd sizes: forward, then all gradients
        dict(name="ffn train odd", op="ffn_train", tokens=501, model=509, hidden=1021, dtype="f32", act="gelu"),
        # a training batch: forward, then all gradients
        dict(name="ffn train batch", op="ffn_train", tokens=4096, model=3584, hidden=18944, dtype="bf16", act="silu"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width over the whole range: often a multiple of 128, sometimes of 8,
    sometimes any number."""
    n = _log_int(rng, lo, hi)
    step = rng.choice((128, 128, 8, 1))
    return max(step, min(hi, n // step * step)) if step > 1 else n


def draw(rng):
    op = rng.choice(("embed", "embed_grad", "norm", "norm_grad", "ffn", "ffn", "ffn_train", "ffn_train"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op in ("embed", "embed_grad"):
        return dict(op=op, tokens=_log_int(rng, 1, 16384), vocab=_log_int(rng, 500, 131072),
                    model=_width(rng, 64, 3584), dtype=dtype, pad=rng.choice((0.0, 0.03, 0.5)))
    if op in ("norm", "norm_grad"):
        return dict(op=op, tokens=_log_int(rng, 1, 16384), model=_width(rng, 64, 8192), dtype=dtype,
                    residual=rng.random() < 0.7)
    model, hidden = _width(rng, 128, 3584), _width(rng, 256, 18944)
    # fp32 products run an order of magnitude slower than half-precision ones
    tokens = _log_int(rng, 1, 4096 if dtype == "bf16" else 1024)
    return dict(op=op, tokens=tokens, model=model, hidden=hidden, dtype=dtype, act=rng.choice(_ACTS))


# ----------------------------------------------------------------- the inputs

def _ids(case, gen, dev):
    """Token ids with a word-like distribution (log-uniform ranks) in a fixed
    scattered order of the vocabulary; a share of them is padding (-1)."""
    v, t = case["vocab"], case["tokens"]
    u = torch.rand(t, generator=gen, device=dev, dtype=torch.float64)
    rank = (torch.exp(u * math.log(v + 1.0)) - 1.0).long().clamp_(0, v - 1)
    ids = (rank * 7919 + 13) % v if v % 7919 else rank
    if case["pad"]:
        ids[torch.rand(t, generator=gen, device=dev) < case["pad"]] = -1
    return ids


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    dt = _DTYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dt)

    op, t, d = case["op"], case["tokens"], case["model"]
    s = {"case": case}
    if op in ("embed", "embed_grad"):
        s["ids"] = _ids(case, gen, dev)
        s["scale"] = math.sqrt(d)
        if op == "embed":
            s["weight"] = normal(case["vocab"], d, std=0.02)
        else:
            s["dy"] = normal(t, d, std=1e-2)
        return s
    if op in ("norm", "norm_grad"):
        # a residual stream's rows differ in size, and a few channels are large
        rows = torch.exp(torch.randn((t, 1), generator=gen, device=dev))
        cols = torch.ones(d, device=dev)
        cols[torch.randint(0, d, (max(1, d // 256),), generator=gen, device=dev)] = 30.0
        s["weight"] = (1.0 + 0.1 * torch.randn(d, generator=gen, device=dev)).to(dt)
        s["x"] = (torch.randn((t, d), generator=gen, device=dev) * rows * cols).to(dt)
        if op == "norm" and case["residual"]:
            s["residual"] = normal(t, d)
        if op == "norm_grad":
            if case["residual"]:  # the gradient that reaches the sum directly
                s["dsum"] = normal(t, d, std=1e-2)
            x = s["x"].float()
            s["rstd"] = torch.rsqrt(x.square().mean(dim=1) + _EPS)
            s["dy"] = normal(t, d, std=1e-2)
        return s
    f = case["hidden"]
    s["x"] = normal(t, d)
    s["w_gate"] = normal(f, d, std=1.0 / math.sqrt(d))
    s["w_up"] = normal(f, d, std=1.0 / math.sqrt(d))
    s["w_down"] = normal(d, f, std=1.0 / math.sqrt(f))
    if op == "ffn_train":
        s["dy"] = normal(t, d, std=1e-2)
    return s


# ------------------------------------------------------------------ one pass

def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if kind == "gelu":
        c = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _DTYPES[case["dtype"]]
    if op == "embed":
        ok = (s["ids"] >= 0) & (s["ids"] < case["vocab"])
        rows = s["weight"][torch.where(ok, s["ids"], 0)].float()
        return (rows * s["scale"] * ok[:, None]).to(dt)
    if op == "embed_grad":
        ok = (s["ids"] >= 0) & (s["ids"] < case["vocab"])
        dw = torch.zeros((case["vocab"], case["model"]), dtype=torch.float32, device=s["dy"].device)
        dw.index_add_(0, torch.where(ok, s["ids"], 0), s["dy"].float() * ok[:, None])
        return (dw * s["scale"]).to(dt)
    if op == "norm":
        v = s["x"].float()
        if case["residual"]:
            v = v + s["residual"].float()
        rstd = torch.rsqrt((v * v).mean(dim=1) + _EPS)
        return {"y": (v * rstd[:, None] * s["weight"].float()).to(dt), "sum": v.to(dt), "rstd": rstd}
    if op == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        n = s["x"].float() * rstd
        wd = dy * s["weight"].float()
        dx = rstd * (wd - n * (wd * n).mean(dim=1, keepdim=True))
        if case["residual"]:
            dx = dx + s["dsum"].float()
        return {"dx": dx.to(dt), "dweight": (dy * n).sum(dim=0).to(dt)}
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(g, case["act"])
    h = a * u
    y = (h @ wd.t()).to(dt)
    if op == "ffn":
        return y
    dy = s["dy"].float()
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return {"y": y, "dx": (dg @ wg + du @ wu).to(dt), "dw_gate": (dg.t() @ x).to(dt),
            "dw_up": (du.t() @ x).to(dt), "dw_down": (dy.t() @ h).to(dt)}


def _own(s):
    import muon_newton_schulz_06_amd as mns
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return mns.muon_embedding(s["ids"], s["weight"], scale=s["scale"])
    if op == "embed_grad":
        return mns.muon_embedding_grad(s["dy"], s["ids"], case["vocab"], scale=s["scale"])
    if op == "norm":
        y, total, rstd = mns.muon_rms_norm(s["x"], s["weight"], residual=s.get("residual"), eps=_EPS)
        return {"y": y, "sum": total, "rstd": rstd}
    if op == "norm_grad":
        dx, dweight = mns.muon_rms_norm_grad(s["dy"], s["x"], s["weight"], s["rstd"], dsum=s.get("dsum"))
        return {"dx": dx, "dweight": dweight}
    w = (s["w_gate"], s["w_up"], s["w_down"])
    if op == "ffn":
        return mns.muon_gated_ffn(s["x"], *w, activation=case["act"])
    y, saved = mns.muon_gated_ffn(s["x"], *w, activation=case["act"], save=True)
    dx, dwg, dwu, dwd = mns.muon_gated_ffn_grad(s["dy"], s["x"], *w, saved)
    return {"y": y, "dx": dx, "dw_gate": dwg, "dw_up": dwu, "dw_down": dwd}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- 64-bit results

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if op in ("embed", "embed_grad"):
        hit = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["vocab"])).squeeze(1)
        if op == "embed":
            y = torch.zeros((case["tokens"], case["model"]), dtype=torch.float64, device=s["ids"].device)
            y[hit] = f64["weight"].index_select(0, s["ids"][hit]) * s["scale"]
            return y
        # runs of equal ids in a stable sorted order, one prefix sum over them
        order = hit[torch.argsort(s["ids"][hit], stable=True)]
        found, count = torch.unique_consecutive(s["ids"][order], return_counts=True)
        dw = torch.zeros((case["vocab"], case["model"]), dtype=torch.float64, device=s["ids"].device)
        if order.numel():
            total = torch.cumsum(f64["dy"][order], dim=0)
            ends = torch.cumsum(count, dim=0)
            sums = total[ends - 1]
            sums[1:] -= total[ends[:-1] - 1]
            dw[found] = sums * s["scale"]
        return dw
    if op == "norm":
        v = f64["x"] + f64["residual"] if case["residual"] else f64["x"]
        r = 1.0 / torch.sqrt(torch.linalg.vecdot(v, v) / case["model"] + _EPS)
        return {"y": v * (r[:, None] * f64["weight"][None, :]), "sum": v, "rstd": r}
    if op == "norm_grad":
        # dx is the vector-Jacobian product of diag(w)·s·r(s), r taken as given
        r, wdy = f64["rstd"], f64["dy"] * f64["weight"]
        along = torch.linalg.vecdot(wdy, f64["x"]) * r * r * r / case["model"]
        dx = wdy * r[:, None] - f64["x"] * along[:, None]
        if case["residual"]:
            dx += f64["dsum"]
        return {"dx": dx, "dweight": (f64["dy"] * f64["x"]).t() @ r}
    wg, wu, wd = f64["w_gate"], f64["w_up"], f64["w_down"]
    gate, up = torch.mm(f64["x"], wg.t()), torch.mm(f64["x"], wu.t())
    if case["act"] == "silu":
        prob = torch.sigmoid(gate)
        slope = prob + gate * prob * (1.0 - prob)
    elif case["act"] == "gelu":
        prob = 0.5 * torch.erfc(-gate / math.sqrt(2.0))
        slope = prob + gate * torch.exp(-gate * gate / 2.0) / math.sqrt(2.0 * math.pi)
    else:
        inner = 2.0 * math.sqrt(2.0 / math.pi)
        prob = torch.sigmoid(inner * (gate + 0.044715 * gate ** 3))  # (1 + tanh(z)) / 2 = sigmoid(2 z)
        slope = prob + gate * prob * (1.0 - prob) * inner * (1.0 + 0.134145 * gate ** 2)
    value = gate * prob
    hidden = value * up
    y = torch.mm(hidden, wd.t())
    if op == "ffn":
        return y
    back = torch.mm(f64["dy"], wd)
    d_up, d_gate = back * value, back * up * slope
    return {"y": y, "dx": torch.mm(d_gate, wg).addmm_(d_up, wu), "dw_gate": torch.mm(d_gate.t(), f64["x"]),
            "dw_up": torch.mm(d_up.t(), f64["x"]), "dw_down": torch.mm(f64["dy"].t(), hidden)}


# --------------------------------------------------- what a pass cannot avoid

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    op, t, d = case["op"], case["tokens"], case["model"]
    if op == "embed":
        return {"bytes": 8 * t + 2 * t * d * e, "flops": t * d}
    if op == "embed_grad":
        return {"bytes": 8 * t + (t + case["vocab"]) * d * e, "flops": 2 * t * d}
    if op == "norm":  # x (and the residual) read, y (and their sum) written
        tensors = 4 if case["residual"] else 2
        return {"bytes": tensors * t * d * e + d * e + 4 * t, "flops": 4 * t * d}
    if op == "norm_grad":  # dy, the normed sum (and the sum's gradient) read, dx written
        tensors = 4 if case["residual"] else 3
        return {"bytes": tensors * t * d * e + 2 * d * e + 4 * t, "flops": 9 * t * d}
    f = case["hidden"]
    if op == "ffn":
        return {"bytes": (3 * d * f + 2 * t * d) * e, "flops": 6.0 * t * d * f}
    return {"bytes": (6 * d * f + 4 * t * d) * e, "flops": 18.0 * t * d * f}
