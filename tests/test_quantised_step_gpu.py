"""A decode step of one layer on 4-bit weights, as its parts are used together: the precompute quantises every projection,
aq_nvfp4_linear_multi makes q, k and v, aq_kv_write norms, rotates and quantises them, aq_tree_attention reads the cache,
aq_nvfp4_linear projects back and makes the logits, aq_token_logprobs scores the drafts. Each part is held against float64
arithmetic on what it was given; then the step is captured and replayed on other tokens."""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from oracle import nvfp4, serving
from rank_weight_reconstruction_gb300 import synth
from helpers import dev_theta

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, DIM, VOCAB, PAGE, CTX, DRAFTS = 256, 4, 1, 128, 1500, 16, 50, 5
LAYOUT = aq.AQ_SF_128X4


def f64(t):
    return t.double().cpu().numpy()


class Layer:
    def __init__(self):
        make = lambda name, out, inp: aq.Nvfp4Weight(*aq.aq_precompute_nvfp4(dev_theta(synth.make_theta(("quantised step", name), out, inp, 8)), sf_layout=LAYOUT), LAYOUT)  # noqa: E731
        self.qkv = [make("q", HEADS * DIM, HIDDEN), make("k", KV * DIM, HIDDEN), make("v", KV * DIM, HIDDEN)]
        self.o, self.head = make("o", HIDDEN, HEADS * DIM), make("head", VOCAB, HIDDEN)
        g = torch.Generator(device="cuda").manual_seed(2)
        wide = lambda: (0.3 * torch.randn(DIM, generator=g, device="cuda")).to(torch.bfloat16)  # noqa: E731
        self.q_norm, self.k_norm = aq.HeadNorm(wide(), offset=1.0), aq.HeadNorm(wide(), offset=1.0)
        self.rope = aq.rope_frequencies(DIM)
        self.cache = aq.KvCache.empty(8, PAGE, KV, DIM, aq.AQ_KV_E4M3)

    def step(self, x, slots, pos, table, ctx, cu, n, tokens):
        qkv = torch.empty(n, (HEADS + 2 * KV) * DIM, dtype=torch.bfloat16, device="cuda")
        cols = list(qkv.split([HEADS * DIM, KV * DIM, KV * DIM], 1))
        aq.aq_nvfp4_linear_multi(self.qkv, x, ys=cols)
        q, k, v = (c.unflatten(1, (-1, DIM)) for c in cols)
        qn = aq.aq_kv_write(self.cache, k, v, slots, rope=self.rope, pos=pos, q=q, q_norm=self.q_norm, k_norm=self.k_norm)
        a = aq.aq_tree_attention(self.cache, qn, cu, ctx, table, max_q=n, out=torch.empty(n, HEADS, DIM, dtype=torch.bfloat16, device="cuda"))
        y = aq.aq_nvfp4_linear(self.o, a.flatten(1))
        logits = aq.aq_nvfp4_linear(self.head, y)
        return qkv, qn, a, y, logits, aq.aq_token_logprobs(logits, tokens, top=4)


def values(w):
    codes, rows, cols = nvfp4.unpack(w.q.cpu().numpy()), w.q.size(0), w.q.size(1) // 8
    sf = w.sf.cpu().numpy().reshape(-(-rows // 128), -(-cols // 4), 32, 4, 4).transpose(0, 3, 2, 1, 4).reshape(-(-rows // 128) * 128, -1)[:rows, :cols]
    return nvfp4.dequantize(codes, sf, np.float32(w.global_scale.item()))


def product_ok(y, x, w):
    X, W = f64(x), values(w)
    ref, size = X @ W.T, np.abs(X) @ np.abs(W).T
    # bf16 output; fp32 sums; x's own unit under its power of two
    assert (np.abs(f64(y) - ref) <= 2.0 ** -8 * np.abs(ref) + (X.shape[1] + 16) * 2.0 ** -23 * size + 2.0 ** -40 * np.abs(X).max(1, keepdims=True) * np.abs(W).sum(1)).all()


def test_step():
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda n: torch.randn(n, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.randperm(8, generator=g, device="cuda").to(torch.int32)[None]
    place = lambda at: table[0, at // PAGE].long() * PAGE + at % PAGE  # noqa: E731
    before = torch.arange(CTX, device="cuda")
    layer.step(randn(CTX), place(before), before.to(torch.int32), table, i32([0]), i32([0, CTX]), CTX, torch.zeros(CTX, dtype=torch.int32, device="cuda"))
    at = torch.arange(CTX, CTX + DRAFTS, device="cuda")
    x, slots, pos = randn(DRAFTS), place(at), at.to(torch.int32)
    tokens = i32([3, 1499, -1, 0, 700])
    args = (x, slots, pos, table, i32([CTX]), i32([0, DRAFTS]), DRAFTS, tokens)

    def check(qkv, qn, a, y, logits, s):
        q, k, v = qkv.split([HEADS * DIM, KV * DIM, KV * DIM], 1)
        for out, w in zip((q, k, v), layer.qkv):
            product_ok(out, x, w)
        angles, _ = serving.rope_angles(DIM)
        for got, flat, norm in ((qn, q, layer.q_norm), (aq.aq_kv_read(layer.cache, slots)[0], k, layer.k_norm)):
            ref = serving.head_norm_rope(f64(flat.unflatten(1, (-1, DIM))), f64(norm.weight), f64(pos), angles, 1e-6, 1.0)
            # queries bf16; keys E4M3: half a step of 2^-3 at most, and what they are read back in
            rel, low = (2.0 ** -8, 1e-5) if got is qn else (2.0 ** -4 + 2.0 ** -7, 2.0 ** -10 / 448 * 1.01)
            assert (np.abs(f64(got) - ref) <= rel * np.abs(ref) + low * np.abs(ref).max(-1, keepdims=True)).all()
        keys, vals = (f64(t)[:, 0] for t in aq.aq_kv_read(layer.cache, place(torch.arange(CTX + DRAFTS, device="cuda"))))
        for i in range(DRAFTS):
            for h in range(HEADS):
                o, _, size = serving.attention_row(f64(qn[i, h]), keys, vals, serving.seen_keys(CTX, DRAFTS, i), DIM ** -0.5)
                # bf16 output; keys and values read back are rounded to bf16 once more than the kernel's: 2^-8 of every logit's terms
                # (norms of heads near sqrt(DIM): |q||k| / sqrt(DIM) below 20) and of every value
                assert (np.abs(f64(a[i, h]) - o) <= 2.0 ** -8 * np.abs(o) + (2 * 20 + 1) * 2.0 ** -8 * size).all()
        product_ok(y, a.flatten(1), layer.o)
        product_ok(logits, y, layer.head)
        lp, lse, hh, tl, tt = serving.token_scores(f64(logits), tokens.cpu().numpy(), 1.0, 4)
        assert np.array_equal(s.top_token.cpu().numpy(), tt)
        for got, ref in ((s.logprob, lp), (s.lse, lse), (s.entropy, hh), (s.top_logprob, tl)):
            assert np.abs(f64(got) - ref).max() <= 1e-3      # (8 x 30 + 16 + 1500) 2^-24 (1 + entropy), below 1e-3

    check(*layer.step(*args))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(*args)
    for _ in range(2):
        x.copy_(randn(DRAFTS))
        tokens.copy_(torch.randint(0, VOCAB, (DRAFTS,), generator=g, device="cuda", dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        check(*out)
    assert aq.aq_device_status() == aq.AQ_OK
