"""One serving step of a decoder that checks drafted tokens, through the library's operators.

Per layer: RMS norm to 8 bits, the 8-bit query/key/value product, attention of the token tree over
the paged cache, the 8-bit output product, and the RMS norm in front of the activation-sparse
FFN. After the last layer the 8-bit vocabulary product gives every node's logits, the drafted tokens
are checked, and the accepted path's keys and values enter the caches. The FFN layers are the
synthetic ones of ``synth``; all other weights are random.

    python examples/draft_step.py          # needs an MI355X and the built library
"""
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import activation_sparse_ffn_layer_amd as pi  # noqa: E402
from synth import CONFIGS, make_layer  # noqa: E402

F16, I32 = torch.float16, torch.int32


def quantize_rows(w):
    """(int8 rows, one scale per row) of a float matrix."""
    scale = (w.abs().amax(1) / 127).clamp(min=1e-12)
    return torch.round(w / scale[:, None]).to(torch.int8), scale


class Decoder:
    """A small decoder: ``layers`` layers of width d around sparse FFNs, ``nodes`` drafted nodes for each
    of ``batch`` sequences per step, a paged cache of ``pages`` pages per layer. It works on the stream that
    is current when it is made: torch's steps between the operators have to run there too."""

    def __init__(self, layers=2, d=1024, heads=16, kv_heads=4, vocab=8000, batch=2, nodes=8, page=16, pages=64, seed=0,
                 device="cuda"):
        g = torch.Generator(device).manual_seed(seed)
        randn = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.d, self.heads, self.kv_heads, self.dim, self.vocab = d, heads, kv_heads, d // heads, vocab
        self.batch, self.nodes, self.T, self.device = batch, nodes, batch * nodes, device
        cfg = dataclasses.replace(CONFIGS["opt6.7b"], d=d, ffn=4 * d, rank=512)
        self.ctx = pi.Context(max_batch=self.T, max_d=d, max_ffn=cfg.ffn, max_rank=cfg.rank)
        qkv = (heads + 2 * kv_heads) * self.dim
        product = lambda n, k: pi.Linear(self.ctx, *quantize_rows(randn(n, k) / k ** 0.5), max_tokens=self.T)  # noqa: E731
        self.embed = randn(vocab, d).to(F16)
        self.layers = []
        for i in range(layers):
            cache = pi.KvCache(self.ctx, *(torch.zeros(pages, page, kv_heads, self.dim, dtype=F16, device=device) for _ in range(2)))
            self.layers.append(dict(
                norm1=1 + 0.1 * randn(d), norm2=1 + 0.1 * randn(d), qkv=product(qkv, d), out=product(d, d), cache=cache,
                attn=pi.Attn(self.ctx, cache, heads, batch, nodes), ffn=pi.Ffn(self.ctx, make_layer(cfg, i, device=device)),
                new=torch.empty(batch, nodes, heads + 2 * kv_heads, self.dim, dtype=F16, device=device)))
        self.norm = 1 + 0.1 * randn(d)
        self.head = product(vocab, d)
        self.verifier = pi.Verifier(self.ctx, vocab, batch, nodes)
        self.len = torch.zeros(batch, dtype=I32, device=device)
        self.table = torch.randperm(pages, generator=g, device=device)[:batch * (pages // batch)].to(I32).view(batch, -1).contiguous()
        empty = lambda *s, dtype=F16: torch.empty(*s, dtype=dtype, device=device)  # noqa: E731
        self.h, self.y = empty(self.T, d), empty(self.T, d)
        self.q8, self.scale = empty(self.T, d, dtype=torch.int8), empty(self.T, dtype=torch.float32)
        self.att, self.o = empty(batch, nodes, heads, self.dim), empty(self.T, d)
        self.f = empty(self.T, d, dtype=torch.float32)
        self.logits = empty(batch, nodes, vocab)
        self.path, self.out = empty(batch, nodes, dtype=I32), empty(batch, nodes, dtype=I32)
        self.count = empty(batch, dtype=I32)

    def forward(self, tokens, tree):
        """Logits [batch][nodes][vocab] of every node of the trees (``tree``: int64 mask words)."""
        c, T, H = self.ctx, self.T, self.heads
        x = self.embed[tokens.long()].view(T, self.d)
        res = None  # the first norm starts the residual
        for l in self.layers:
            pi.add_rmsnorm(c, x, res, l["norm1"], 1e-5, self.h, q=self.q8, scale=self.scale)
            pi.linear_q8(c, l["qkv"], self.q8, self.scale, l["new"].view(T, -1))
            q, k, v = l["new"].split([H, self.kv_heads, self.kv_heads], 2)
            pi.tree_attention(c, l["attn"], q, k, v, tree, self.table, self.len, self.att)
            a = self.att.view(T, self.d)
            # the 8-bit product takes 8-bit rows: those of the attention's output without a norm's weight
            s = (a.float().abs().amax(1) / 127).clamp(min=1e-12)
            pi.linear_q8(c, l["out"], torch.round(a.float() / s[:, None]).to(torch.int8), s, self.o)
            pi.add_rmsnorm(c, self.o, self.h, l["norm2"], 1e-5, self.h, y=self.y)
            pi.layer(c, l["ffn"], self.y, self.f)
            x, res = self.f, self.h
        pi.add_rmsnorm(c, x, res, self.norm, 1e-5, self.h, q=self.q8, scale=self.scale)
        pi.linear_q8(c, self.head, self.q8, self.scale, self.logits.view(T, self.vocab))
        return self.logits

    def step(self, tokens, parents, tree, u, u_next, q=None, temperature=None):
        """Check the drafted trees and keep the accepted paths: (nodes, tokens, counts)."""
        self.forward(tokens, tree)
        pi.verify(self.ctx, self.verifier, self.logits, tokens, parents, u, u_next, self.path, self.out, self.count, q=q,
                  temperature=temperature)
        for i, l in enumerate(self.layers):
            _, k, v = l["new"].split([self.heads, self.kv_heads, self.kv_heads], 2)
            last = i + 1 == len(self.layers)
            pi.kv_append(self.ctx, l["cache"], k, v, self.table, self.len, self.len if last else None, self.path, self.count)
        return self.path, self.out, self.count


def ancestors(parents):
    """int64 mask words [B][N]: bit j of node i where j is i or above it."""
    rows = []
    for par in parents.tolist():
        w = []
        for i, p in enumerate(par):
            w.append((w[p] if p >= 0 else 0) | 1 << i)
        rows.append([x - (1 << 64) if x >= 1 << 63 else x for x in w])
    return torch.tensor(rows, dtype=torch.int64, device=parents.device)


def main():
    dec = Decoder()
    g = torch.Generator("cuda").manual_seed(1)
    parents = torch.tensor([[-1, 0, 0, 1, 1, 2, 3, 5]] * dec.batch, dtype=I32, device="cuda")
    tree = ancestors(parents)
    last = torch.randint(0, dec.vocab, (dec.batch, 1), generator=g, device="cuda").to(I32)
    for step in range(8):
        drafted = torch.randint(0, dec.vocab, (dec.batch, dec.nodes - 1), generator=g, device="cuda").to(I32)
        u = torch.rand(dec.batch, dec.nodes, generator=g, device="cuda")
        path, out, n = dec.step(torch.cat([last, drafted], 1), parents, tree, u, u[:, 0].contiguous(),
                                temperature=torch.full((dec.batch,), 0.8, device="cuda"))
        last = torch.take_along_dim(out, n.long()[:, None] - 1, 1)
        print(f"step {step}: kept {n.tolist()} tokens, next {last.flatten().tolist()}, cache lengths {dec.len.tolist()}")


if __name__ == "__main__":
    main()
