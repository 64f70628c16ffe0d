"""Trains a small next-token model made of the library's layers, its
feed-forward matrices with Muon:

    ids → Embedding → N × [ s = s + y; n = RMSNorm(s); y = GatedFFN(n) ]
        → RMSNorm → logits (tied to the embedding) → cross entropy

    python examples/train_ffn_lm.py [--steps 60] [--tokens 4096] [--dtype bf16]

The data is synthetic: a fixed random successor for every token, with noise,
so that the model (which mixes no positions) can learn it.  Muon takes the
feed-forward matrices, AdamW the embedding and the norms' weights.  The logits
and the loss are plain torch.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import muon_newton_schulz_06_amd as mns  # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, vocab, model, hidden, depth, **kw):
        super().__init__()
        self.embedding = mns.Embedding(vocab, model, scale=model ** 0.5, **kw)
        self.norms = torch.nn.ModuleList(mns.RMSNorm(model, **kw) for _ in range(depth + 1))
        self.blocks = torch.nn.ModuleList(mns.GatedFFN(model, hidden, **kw) for _ in range(depth))

    def forward(self, ids):
        s = self.embedding(ids)
        y = None
        for norm, block in zip(self.norms, self.blocks):
            if y is None:
                n = norm(s)
            else:  # the residual's addition and the norm in one kernel
                n, s = norm(y, s)
            y = block(n)
        n, _ = self.norms[-1](y, s)
        return n @ self.embedding.weight.t()


def train(steps=60, tokens=4096, vocab=2048, model=512, hidden=1536, depth=2, dtype=torch.bfloat16, seed=0,
          log=print):
    """Returns the losses of all steps."""
    torch.manual_seed(seed)
    dev = torch.device("cuda")
    net = Model(vocab, model, hidden, depth, device=dev, dtype=dtype)
    matrices = [p for b in net.blocks for p in b.parameters()]
    rest = [net.embedding.weight] + [n.weight for n in net.norms]
    optimisers = [mns.Muon(matrices, lr=0.02), torch.optim.AdamW(rest, lr=3e-3, weight_decay=0.0)]
    gen = torch.Generator(device=dev).manual_seed(seed + 1)
    successor = torch.randperm(vocab, generator=gen, device=dev)
    losses = []
    began = time.perf_counter()
    for step in range(steps):
        ids = torch.randint(0, vocab, (tokens,), generator=gen, device=dev)
        noise = torch.rand(tokens, generator=gen, device=dev) < 0.1
        target = torch.where(noise, torch.randint(0, vocab, (tokens,), generator=gen, device=dev), successor[ids])
        loss = torch.nn.functional.cross_entropy(net(ids).float(), target)
        loss.backward()
        for o in optimisers:
            o.step()
            o.zero_grad(set_to_none=True)
        losses.append(loss.detach())
        if step % 10 == 0 or step == steps - 1:
            log(f"step {step:4d}  loss {float(losses[-1]):.4f}  {(time.perf_counter() - began) / (step + 1) * 1e3:.2f} ms per step")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--dtype", choices=("bf16", "f32"), default="bf16")
    a = ap.parse_args()
    out = train(a.steps, a.tokens, dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32)
    if not out[-1] < out[0]:
        raise SystemExit("the loss did not fall")
