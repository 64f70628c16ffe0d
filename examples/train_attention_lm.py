"""Trains a small language model of the library's layers on a packed batch of
documents, its matrices with Muon:

    ids → Embedding → N × [ x = x + drop(DiffAttention(Rotary(RMSNorm(x)·W)) · W)
                            x = x + drop(GatedFFN(RMSNorm(x))) ]
        → RMSNorm → logits (tied to the embedding) → cross entropy

    python examples/train_attention_lm.py [--steps 60] [--tokens 4096] [--dtype bf16]

The data is synthetic: every document repeats a random phrase of its own, so
that the model, which has to look back for the phrase, can learn it.  Muon takes
the matrices, AdamW the embedding, the norms' weights and λ's vectors.  The
projections, logits and loss are plain torch.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import muon_newton_schulz_06_amd as mns  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, heads, kv_heads, dim, hidden, layer, dropout, **kw):
        super().__init__()
        model = 2 * heads * dim
        self.sizes = (2 * heads, 2 * kv_heads, kv_heads, dim)
        self.qkv = torch.nn.Linear(model, (2 * heads + 4 * kv_heads) * dim, bias=False, **kw)
        self.out = torch.nn.Linear(model, model, bias=False, **kw)
        self.rotary = mns.Rotary(dim)
        # λ begins smaller in the first layers
        init = 0.8 - 0.6 * 2.718281828459045 ** (-0.3 * layer)
        self.attention = mns.DiffAttention(heads, dim, kv_heads, lambda_init=init, **kw)
        self.norms = torch.nn.ModuleList(mns.RMSNorm(model, **kw) for _ in range(2))
        self.ffn = mns.GatedFFN(model, hidden, **kw)
        self.drops = torch.nn.ModuleList(mns.Dropout(dropout, seed=2 * layer + i, device=kw.get("device")) for i in range(2))

    def forward(self, x, offsets, positions):
        tokens, (q, k, v, dim) = x.shape[0], self.sizes
        heads = self.qkv(self.norms[0](x)).view(tokens, -1, dim)
        values = heads[:, q + k:].reshape(tokens, v, 2 * dim)
        a, b = self.rotary(heads[:, :q], heads[:, q:q + k], positions)
        y = self.attention(a, b, values, offsets)
        x = self.drops[0](self.out(y.reshape(tokens, -1)), x)
        return self.drops[1](self.ffn(self.norms[1](x)), x)


class Model(torch.nn.Module):
    def __init__(self, vocab, heads, kv_heads, dim, hidden, depth, dropout=0.1, **kw):
        super().__init__()
        model = 2 * heads * dim
        self.embedding = mns.Embedding(vocab, model, scale=model ** 0.5, **kw)
        self.blocks = torch.nn.ModuleList(Block(heads, kv_heads, dim, hidden, i, dropout, **kw) for i in range(depth))
        self.norm = mns.RMSNorm(model, **kw)

    def forward(self, ids, offsets, positions):
        x = self.embedding(ids)
        for block in self.blocks:
            x = block(x, offsets, positions)
        return self.norm(x) @ self.embedding.weight.t()


def batch(tokens, documents, vocab, gen, dev):
    """(ids, offsets, positions): documents of random lengths, each a phrase of
    4 to 16 tokens over and over."""
    cuts = torch.randperm(tokens - 1, generator=gen, device=dev)[:documents - 1].sort().values + 1
    ends = torch.tensor([0, tokens], device=dev)
    offsets = torch.cat([ends[:1], cuts, ends[1:]]).int()
    document = torch.bucketize(torch.arange(tokens, device=dev), cuts, right=True)
    positions = torch.arange(tokens, device=dev) - offsets[document]
    phrase = torch.randint(0, vocab, (documents, 16), generator=gen, device=dev)
    length = torch.randint(4, 17, (documents,), generator=gen, device=dev)
    return phrase[document, positions % length[document]], offsets, positions


def train(steps=60, tokens=4096, documents=24, vocab=512, heads=4, kv_heads=2, dim=64, hidden=1536, depth=2, dropout=0.1,
          dtype=torch.bfloat16, seed=0, log=print):
    """Returns the losses of all steps."""
    torch.manual_seed(seed)
    dev = torch.device("cuda")
    net = Model(vocab, heads, kv_heads, dim, hidden, depth, dropout, device=dev, dtype=dtype)
    matrices = [p for b in net.blocks for p in b.parameters() if p.dim() == 2]
    rest = [p for p in net.parameters() if not any(p is m for m in matrices)]
    optimisers = [mns.Muon(matrices, lr=0.02), torch.optim.AdamW(rest, lr=3e-3, weight_decay=0.0)]
    gen = torch.Generator(device=dev).manual_seed(seed + 1)
    losses = []
    began = time.perf_counter()
    for step in range(steps):
        ids, offsets, positions = batch(tokens, documents, vocab, gen, dev)
        logits = net(ids, offsets, positions).float()
        # the next token; a document's last has none
        target = torch.roll(ids, -1).index_fill(0, offsets[1:].long() - 1, -100)
        loss = torch.nn.functional.cross_entropy(logits, target)
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
    train(a.steps, a.tokens, dtype=torch.bfloat16 if a.dtype == "bf16" else torch.float32)
