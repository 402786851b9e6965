"""One step of tree-drafted decoding with every projection a reconstruction linear.

A small model of the Gemma-3-1B layer's shapes (hidden 1152, four query heads and one key/value head of 256,
MLP 6912) runs a tree of drafted tokens in one pass: the projections through aq_linear_qkv, aq_linear and
aq_mlp, positions and the quantised cache through aq_kv_write, attention through aq_tree_attention, and at
the end aq_verify_drafts accepts a path of the tree and draws the token after it. Weights are synthetic.

    python examples/draft_tree_step.py
"""
from __future__ import annotations

import os
import sys
from dataclasses import dataclass

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import rank_weight_reconstruction_gb300 as aq  # noqa: E402
from rank_weight_reconstruction_gb300 import synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, INTER, RANK = 1152, 4, 1, 256, 6912, 16
PAGE = 64


def theta(key, out, inp):
    """A seeded bundle on the device."""
    t = synth.make_theta(key, out, inp, RANK)
    dev = lambda bits: torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).cuda()  # noqa: E731
    return aq.Theta(W0=dev(t.W0)[:, :inp], s=dev(t.s), U=dev(t.U)[:, :RANK], V=dev(t.V)[:, :RANK])


@dataclass
class Layer:
    qkv: list
    o: object
    gate: object
    up: object
    down: object
    cache: object
    window: int


class Model:
    """`layers` layers, every second one with a sliding window; `pages` pages of cache a layer."""

    def __init__(self, layers: int = 2, vocab: int = 4096, pages: int = 16, kind: int = aq.AQ_KV_E4M3, window: int = 32):
        self.layers = []
        for l in range(layers):
            f = lambda name, out, inp: theta(("draft-tree", l, name), out, inp)  # noqa: E731
            self.layers.append(Layer(
                qkv=[f("q", HEADS * DIM, HIDDEN), f("k", KV_HEADS * DIM, HIDDEN), f("v", KV_HEADS * DIM, HIDDEN)],
                o=f("o", HIDDEN, HEADS * DIM), gate=f("gate", INTER, HIDDEN), up=f("up", INTER, HIDDEN),
                down=f("down", HIDDEN, INTER), cache=aq.KvCache.empty(pages, PAGE, KV_HEADS, DIM, kind),
                window=window if l % 2 else 0))
        g = torch.Generator(device="cuda").manual_seed(1)
        self.embed = torch.randn(vocab, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)
        self.rope = aq.rope_frequencies(DIM)

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def forward(self, tokens, ctx, table, cu, max_q, depth=None, mask=None):
        """Hidden states [total, HIDDEN] of the batch's newest tokens: ctx int32 [batch] tokens lie in the caches
        already; the tree's keys and values go behind them, token by token in index order."""
        seq = torch.repeat_interleave(torch.arange(ctx.numel(), device="cuda"), (cu[1:] - cu[:-1]).long())
        index = torch.arange(tokens.numel(), device="cuda") - cu[:-1].long()[seq]          # within the sequence
        at = ctx.long()[seq] + index                                                       # place in the cache
        slots = table.long()[seq, at // PAGE] * PAGE + at % PAGE
        pos = (ctx.long()[seq] + (index if depth is None else depth.long())).to(torch.int32)
        x = self.embed[tokens]
        for layer in self.layers:
            qkv = torch.empty(tokens.numel(), (HEADS + 2 * KV_HEADS) * DIM, dtype=torch.bfloat16, device="cuda")
            cols = [qkv[:, :HEADS * DIM], qkv[:, HEADS * DIM:(HEADS + KV_HEADS) * DIM], qkv[:, (HEADS + KV_HEADS) * DIM:]]
            aq.aq_linear_qkv(layer.qkv, self.norm(x), ys=cols)
            q, k, v = (c.unflatten(1, (-1, DIM)) for c in cols)
            aq.aq_kv_write(layer.cache, k, v, slots, rope=self.rope, pos=pos, q=q, q_out=q)
            a = aq.aq_tree_attention(layer.cache, q, cu, ctx, table, max_q=max_q, mask=mask, depth=depth,
                                     window=layer.window, out=torch.empty_like(q, memory_format=torch.contiguous_format))
            x = x + aq.aq_linear(layer.o, a.flatten(1))
            x = x + aq.aq_mlp(layer.gate, layer.up, layer.down, self.norm(x))
        return self.norm(x)

    def probabilities(self, hidden):
        return torch.softmax(hidden.float() @ self.embed.float().T / HIDDEN ** 0.5, -1)


def tree_mask(parent):
    """Ancestor bits (int64 [n, 1], n <= 64) and depths (int32 [n]) of one tree."""
    bits, depth = [], []
    for i, p in enumerate(parent):
        bits.append((1 << i) | (bits[p] if p >= 0 else 0))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    signed = [b - (1 << 64) if b >> 63 else b for b in bits]
    return torch.tensor(signed, dtype=torch.int64, device="cuda")[:, None], torch.tensor(depth, dtype=torch.int32, device="cuda")


def step(model, prompt, drafts, parent, seed: int = 0):
    """Prefills `prompt` (all but its last token), then runs that last token and the drafted tree behind it: row 0 of
    the tree is the last token, draft i is row i + 1. Returns (hidden states of the rows, accepted path, next
    token)."""
    n, ctx = len(drafts), len(prompt) - 1
    table = torch.arange(model.layers[0].cache.k.size(0), dtype=torch.int32, device="cuda")[None]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    tok = torch.tensor(list(prompt) + list(drafts), device="cuda")
    if ctx:
        model.forward(tok[:ctx], i32([0]), table, i32([0, ctx]), ctx)
    mask, depth = tree_mask([-1] + [p + 1 for p in parent])
    hidden = model.forward(tok[ctx:], i32([ctx]), table, i32([0, n + 1]), n + 1, depth=depth, mask=mask)
    g = torch.Generator(device="cuda").manual_seed(seed)
    noise = torch.empty(1, model.embed.size(0), device="cuda").exponential_(generator=g).clamp_(min=1e-10)
    count, path, token = aq.aq_verify_drafts(model.probabilities(hidden), i32(list(drafts)), i32([0, n]),
                                             torch.rand(n, generator=g, device="cuda"), noise, parent=i32(list(parent)))
    return hidden, path[0, :int(count[0])].tolist(), int(token[0])


def main():
    model = Model()
    prompt = [int(t) for t in np.random.RandomState(0).randint(0, 4096, 100)]
    # three guesses for the next token, two for the one after each of the first two, and so on
    parent = [-1, -1, -1, 0, 0, 1, 1, 3, 3, 7]
    model_guess = model.forward(torch.tensor(prompt, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"),
                                torch.arange(16, dtype=torch.int32, device="cuda")[None],
                                torch.tensor([0, len(prompt)], dtype=torch.int32, device="cuda"), len(prompt))
    best = model.probabilities(model_guess[-1:])[0].topk(len(parent)).indices.tolist()
    hidden, path, token = step(model, prompt, best, parent)
    print(f"{len(parent)} drafts behind {len(prompt)} tokens: accepted {[best[i] for i in path]}, next token {token}")
    if aq.aq_device_status() != aq.AQ_OK:
        raise SystemExit("device status word reports an expired wait")


if __name__ == "__main__":
    main()
