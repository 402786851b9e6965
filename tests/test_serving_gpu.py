"""The serving operators on the GPU against the float64 oracle (oracle/serving.py).

Tolerances, derived from the formats and the operations (bf16: half an ulp is 2^-8 of the value's power of
two; fp32: 2^-24):
  rotation     one bf16 rounding of the output plus fp32 evaluation of two products and of the angle (a
               float32 argument of at most half a turn: 2^-24 of pi, and two ulp of the sine): in all below
               1e-6 of |a| + |b|
  quantising   half an E4M3 step at the vector's scale plus the bf16 rounding of what is read back
  attention    the output's bf16 rounding, 2^-8 |o|; weights held in 8 bits, 2^-8 of sum p|v| (half as much
               again for the fp32 exp and sums); scores: E4M3 queries keep elements above 2^-18 of the head's
               largest, so a score is off by at most e = 2^-18 max|q| sum|k| scale, plus 2^-20 of sum|q||k|
               scale for the fp32 sums, and a weight by 2e of itself; weights below 2^-18 of a tile's largest
               are lost: 2^-17 max|v|
  verification whole numbers, compared exactly on inputs whose closest comparison is 1e-5 from a tie
"""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from oracle import serving

pytestmark = pytest.mark.gpu

DT = {"bf16": aq.AQ_KV_BF16, "e4m3": aq.AQ_KV_E4M3}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def randn(r, *shape):
    return torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(torch.bfloat16).cuda()


# ------------------------------------------------------------------------------------------
# rotary positions
# ------------------------------------------------------------------------------------------
RULES = {"none": aq.AQ_ROPE_SCALE_NONE, "linear": aq.AQ_ROPE_SCALE_LINEAR, "ntk": aq.AQ_ROPE_SCALE_NTK,
         "yarn": aq.AQ_ROPE_SCALE_YARN, "wavelength": aq.AQ_ROPE_SCALE_WAVELENGTH}


def rope_ok(got, x, pos, angles, mag, layout, inverse=False):
    ref = serving.rope(x, pos, angles, mag, layout, inverse)
    n = len(angles)
    size = np.zeros_like(ref)
    lo = slice(0, n) if layout == "half" else slice(0, 2 * n, 2)
    hi = slice(n, 2 * n) if layout == "half" else slice(1, 2 * n, 2)
    size[..., lo] = size[..., hi] = (np.abs(x[..., lo]) + np.abs(x[..., hi])) * mag
    d = np.abs(got - ref)
    bad = d > 2.0 ** -8 * np.abs(ref) + 1e-6 * size
    assert not bad.any(), (float(d.max()), np.argwhere(bad)[:4])


@pytest.mark.parametrize("T,H,D,rot,layout,rule", [
    (1, 1, 16, 16, "half", "none"), (1, 4, 256, 256, "half", "none"), (5, 3, 64, 16, "interleaved", "linear"),
    (33, 7, 80, 48, "half", "yarn"), (130, 2, 128, 128, "interleaved", "wavelength"), (257, 5, 96, 96, "half", "ntk"),
    (1000, 16, 128, 64, "half", "none"), (3000, 32, 128, 128, "half", "none"), (3001, 33, 64, 64, "interleaved", "none"),
])
def test_rope_matches_oracle(T, H, D, rot, layout, rule):
    r = np.random.RandomState(T + H + D)
    code = aq.AQ_ROPE_HALF if layout == "half" else aq.AQ_ROPE_INTERLEAVED
    rope = aq.rope_frequencies(rot, scaling=RULES[rule], factor=4.0, original_len=2048, layout=code)
    angles, mag = serving.rope_angles(rot, rule=rule, factor=4.0, original_len=2048)
    x = randn(r, T, H, D)
    pos = r.randint(-5, 1 << 20, T).astype(np.int32)
    pos[0], pos[-1] = 0, 2 ** 31 - 1
    p = torch.from_numpy(pos).cuda()
    rope_ok(f64(aq.aq_rope(rope, p, x)), f64(x), pos, angles, mag, layout)
    back = aq.aq_rope(rope, p, x, inverse=True)
    rope_ok(f64(back), f64(x), pos, angles, mag, layout, inverse=True)


def test_rope_inverse_is_the_gradient():
    """The inverse applied to an output gradient against central differences of <g, rope(x)> in the oracle's
    float64, and against the transpose of the formula."""
    r = np.random.RandomState(3)
    x, g, pos = randn(r, 2, 1, 32), randn(r, 2, 1, 32), np.array([5, 77], np.int32)
    rope = aq.rope_frequencies(32)
    angles, mag = serving.rope_angles(32)
    got = f64(aq.aq_rope(rope, torch.from_numpy(pos).cuda(), g, inverse=True))
    X, G, h = f64(x), f64(g), 1e-4
    for t in range(2):
        for i in range(32):
            up, dn = X.copy(), X.copy()
            up[t, 0, i] += h
            dn[t, 0, i] -= h
            diff = ((serving.rope(up, pos, angles) - serving.rope(dn, pos, angles)) * G).sum() / (2 * h)
            # bf16 rounding of the gradient, and the differences' own 1e-8
            assert abs(got[t, 0, i] - diff) <= 2.0 ** -8 * abs(diff) + 1e-5, (t, i)


def test_rope_strides_in_place_and_streams():
    r = np.random.RandomState(4)
    T, H, D = 37, 6, 64
    rope = aq.rope_frequencies(64)
    angles, mag = serving.rope_angles(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 100
    packed = randn(r, T, 3 * H * D)
    x = packed[:, H * D:2 * H * D].unflatten(1, (H, D))          # column slice of a stacked output
    want = f64(x).copy()
    before = packed.clone()
    y = torch.full((H, T, D), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    aq.aq_rope(rope, pos, x, y=y)                                  # heads outermost
    rope_ok(f64(y), want, pos.cpu().numpy(), angles, mag, "half")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    aq.aq_rope(rope, pos, x, y=x, stream=side)                     # in place, on another stream
    side.synchronize()
    rope_ok(f64(x), want, pos.cpu().numpy(), angles, mag, "half")
    packed[:, H * D:2 * H * D] = before[:, H * D:2 * H * D]
    assert torch.equal(packed, before)                             # nothing else was touched
    assert aq.aq_rope(rope, pos[:0], x[:0]).shape == (0, H, D)


# ------------------------------------------------------------------------------------------
# the cache
# ------------------------------------------------------------------------------------------
def quantised(x):
    """Codes' values and scales by the documented rule in fp32 (what the kernel computes, bit for bit)."""
    x = x.float()
    scale = torch.clamp(x.abs().amax(-1) * torch.tensor(1.0 / 448.0, dtype=torch.float32), min=2.0 ** -100)
    code = torch.clamp(x * (1.0 / scale)[..., None], -448, 448).to(torch.float8_e4m3fn).float()
    return code, scale


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("T,hq,hk,D,page", [(1, 4, 1, 256, 16), (7, 8, 2, 128, 64), (65, 3, 3, 80, 128),
                                            (1030, 2, 2, 16, 32), (2500, 32, 8, 64, 256)])
def test_kv_write_and_read(kind, T, hq, hk, D, page):
    r = np.random.RandomState(T)
    pages = -(-T // page) + 2
    cache = aq.KvCache.empty(pages, page, hk, D, DT[kind])
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.fill_(7)
    qkv = randn(r, T, (hq + 2 * hk) * D)
    q, k, v = (qkv[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    slots = torch.from_numpy(r.permutation(pages * page)[:T].astype(np.int64)).cuda()
    pos = torch.from_numpy(r.randint(0, 40000, T).astype(np.int32)).cuda()
    rope, (angles, mag) = aq.rope_frequencies(D), serving.rope_angles(D)
    q_out = aq.aq_kv_write(cache, k, v, slots, rope=rope, pos=pos, q=q)
    rope_ok(f64(q_out), f64(q), pos.cpu().numpy(), angles, mag, "half")
    kb, vb = aq.aq_kv_read(cache, slots)
    turned = serving.rope(f64(k), pos.cpu().numpy(), angles, mag)
    if kind == "bf16":
        assert torch.equal(vb, v)
        rope_ok(f64(kb), f64(k), pos.cpu().numpy(), angles, mag, "half")
    else:
        code, scale = quantised(v)
        assert torch.equal(vb, (code * scale[..., None]).to(torch.bfloat16))
        amax = np.abs(turned).max(-1, keepdims=True)
        unit = amax / 448.0
        val = np.abs(turned) / unit
        step = 2.0 ** (np.floor(np.log2(np.maximum(val, 2.0 ** -6))) - 3)
        assert np.all(np.abs(f64(kb) - turned) <= (0.5 * step * unit + 2.0 ** -8 * np.abs(f64(kb))) * 1.001 + 2e-6 * amax)
    # untouched slots keep what they held
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[slots] = False
    cells = cache.v.transpose(1, 2).reshape(pages * page, hk, D)[rest]
    assert bool((cells.float() == 7).all())
    if kind == "e4m3":
        assert bool((cache.k_scale.transpose(1, 2).reshape(pages * page, hk)[rest] == 7).all())


def test_kv_special_vectors_and_slots():
    """Zeros, subnormals, the largest bf16, infinities and NaN; slots outside the cache."""
    D, page = 64, 16
    cache = aq.KvCache.empty(2, page, 1, D, aq.AQ_KV_E4M3)
    cache.k.fill_(0x7f)
    cache.k_scale.fill_(float("nan"))
    x = torch.zeros(8, 1, D, dtype=torch.float32)
    x[1, 0, 5] = 1e-39
    x[2] = 3e38
    x[3, 0, 0] = float("inf")
    x[4, 0, 63] = float("nan")
    x[5] = torch.linspace(-1, 1, D)
    x[6], x[7] = 1.0, 2.0
    x = x.to(torch.bfloat16).cuda()
    slots = torch.tensor([0, 1, 2, 3, 4, 31, -1, 32], dtype=torch.int64, device="cuda")
    aq.aq_kv_write(cache, x, x, slots)
    k, v = aq.aq_kv_read(cache, slots)
    assert torch.equal(k[0], x[0]) and not k[1].any()
    assert torch.equal(k[2], x[2]) and torch.isnan(k[3]).all() and torch.isnan(k[4]).all()
    code, scale = quantised(x[5])
    assert torch.equal(k[5], (code * scale[..., None]).to(torch.bfloat16))
    assert not k[6:].any() and not v[6:].any()                   # outside the cache: zeros
    assert bool(((cache.k & 0x7f) != 0x7f).all(-1).view(2, page)[0, :5].all())   # codes stay finite
    assert bool((cache.k[0, 0, 5:] == 0x7f).all())


def test_kv_write_in_place_queries_and_layouts():
    r = np.random.RandomState(8)
    T, hq, hk, D, page = 21, 4, 2, 128, 16
    cache = aq.KvCache.empty(4, page, hk, D, aq.AQ_KV_BF16)
    qkv = randn(r, T, (hq + 2 * hk) * D)
    before = qkv.clone()
    q, k, v = (qkv[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, 4), (4, 6), (6, 8)))
    slots = torch.arange(5, 5 + T, device="cuda")
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope = aq.rope_frequencies(64, layout=aq.AQ_ROPE_INTERLEAVED)
    angles, mag = serving.rope_angles(64)
    aq.aq_kv_write(cache, k, v, slots, rope=rope, pos=pos, q=q, q_out=q)
    rope_ok(f64(q), f64(before)[:, :hq * D].reshape(T, hq, D), pos.cpu().numpy(), angles, mag, "interleaved")
    assert torch.equal(qkv[:, hq * D:], before[:, hq * D:])
    out = torch.empty(T, 2 * hk * D, dtype=torch.bfloat16, device="cuda")
    kb, vb = out[:, :hk * D].unflatten(1, (hk, D)), out[:, hk * D:].unflatten(1, (hk, D))
    aq.aq_kv_read(cache, slots, k=kb, v=vb)
    assert torch.equal(vb, v)
    rope_ok(f64(kb), f64(k), pos.cpu().numpy(), angles, mag, "interleaved")


# ------------------------------------------------------------------------------------------
# attention
# ------------------------------------------------------------------------------------------
class Case:
    """A batch of sequences with a cache whose every unnamed cell is NaN."""

    def __init__(self, seed, kind, D, hk, group, page, ctx, drafted, tree="chain", window=0, gain=2.0, v_gain=1.0):
        r = self.r = np.random.RandomState(seed)
        self.kind, self.D, self.hk, self.group, self.page, self.window = kind, D, hk, group, page, window
        self.ctx, self.T, B = list(ctx), list(drafted), len(ctx)
        total = sum(self.T)
        need = [-(-(c + t) // page) for c, t in zip(ctx, drafted)]
        pages = sum(need) + 3
        order = r.permutation(pages)[:sum(need)]
        table = np.full((B, max(max(need), 1) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table_np, self.table = table, torch.from_numpy(table).cuda()
        self.cache = aq.KvCache.empty(pages, page, hk, D, DT[kind])
        for t in (self.cache.k, self.cache.v):
            t.fill_(0x7f if kind == "e4m3" else float("nan"))
        if kind == "e4m3":
            self.cache.k_scale.fill_(float("nan"))
            self.cache.v_scale.fill_(float("inf"))
        slots = np.concatenate([[table[b, j // page] * page + j % page for j in range(c + t)]
                                for b, (c, t) in enumerate(zip(ctx, drafted))] + [np.zeros(0)]).astype(np.int64)
        self.slots = torch.from_numpy(slots).cuda()
        n = len(slots)
        k, v = randn(r, n, hk, D), (randn(r, n, hk, D).float() * v_gain).to(torch.bfloat16)
        if n:
            aq.aq_kv_write(self.cache, k, v, self.slots)
        self.q = (randn(r, total, hk * group, D).float() * gain).to(torch.bfloat16)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.T)]), dtype=torch.int32, device="cuda")
        self.ctx_t = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.max_q = max(self.T)
        self.bits = self.depth = self.mask = None
        if tree != "chain":
            self.bits, self.depth = [], []
            for t in self.T:
                bits, depth = np.zeros((t, t), bool), np.zeros(t, np.int32)
                for i in range(t):
                    par = r.randint(-1, i) if i else -1
                    if par >= 0:
                        bits[i], depth[i] = bits[par], depth[par] + 1
                    bits[i, i] = True
                if tree == "sparse":      # rows that see none of the drafted tokens, not even themselves
                    bits[::2] = False
                self.bits.append(bits)
                self.depth.append(depth)
            words = -(-self.max_q // 64) + 1
            m = np.zeros((total, words), np.uint64)
            at = 0
            for bits in self.bits:
                for i, j in np.argwhere(bits):
                    m[at + i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
                at += len(bits)
            self.mask = torch.from_numpy(m.view(np.int64)).cuda()
            self.depth_t = torch.tensor(np.concatenate(self.depth), dtype=torch.int32, device="cuda")

    def run(self, **kw):
        out, lse = aq.aq_tree_attention(self.cache, self.q, self.cu, self.ctx_t, self.table, max_q=self.max_q,
                                        mask=self.mask, depth=None if self.mask is None else self.depth_t,
                                        window=self.window, return_lse=True, **kw)
        return out, lse

    def keys(self):
        """k and v of every slot in order, in float64, as the cache holds them (codes times scale)."""
        got = []
        for codes, scale in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            flat = codes.transpose(1, 2).reshape(-1, self.hk, self.D)[self.slots]
            if scale is None:
                got.append(f64(flat))
            else:
                s = scale.transpose(1, 2).reshape(-1, self.hk)[self.slots]
                got.append(f64(flat.view(torch.float8_e4m3fn)) * f64(s)[..., None])
        return got

    def check(self, out, lse, rows=None):
        K, V = self.keys()
        Q, O, L = f64(self.q), f64(out), f64(lse)
        scale, at, first = self.D ** -0.5, 0, 0
        for b, (c, t) in enumerate(zip(self.ctx, self.T)):
            # keys in pages the table does not name are left out
            named = self.table_np[b, np.arange(c + t) // self.page] if c + t else np.zeros(0)
            held = (named >= 0) & (named < self.cache.k.size(0))
            for i in range(t):
                if rows is not None and (at + i) not in rows:
                    continue
                seen = held & serving.seen_keys(c, t, i, None if self.bits is None else self.bits[b][i],
                                                None if self.depth is None else self.depth[b], self.window)
                for h in range(self.hk * self.group):
                    k, v, q = K[first:first + c + t, h // self.group], V[first:first + c + t, h // self.group], Q[at + i, h]
                    o, l, a = serving.attention_row(q, k, v, seen, scale)
                    got, where = O[at + i, h], (b, i, h)
                    if not seen.any():
                        assert not got.any() and L[at + i, h] == -np.inf, where
                        continue
                    ks = np.abs(k[seen])
                    e = scale * (2.0 ** -20 * (ks @ np.abs(q)).max()
                                 + (2.0 ** -18 * np.abs(q).max() * ks.sum(-1).max() if self.kind == "e4m3" else 0))
                    tol = 2.0 ** -8 * np.abs(o) + (1.5 * 2.0 ** -8 + 4 * e) * a + 2.0 ** -17 * np.abs(v[seen]).max()
                    assert np.all(np.abs(got - o) <= tol), (where, float(np.abs(got - o).max()), float(tol.min()))
                    assert abs(L[at + i, h] - l) <= e + 2e-5 + 1e-6 * abs(l), (where, L[at + i, h], l)
            at, first = at + t, first + c + t


KINDS = pytest.mark.parametrize("kind", ["bf16", "e4m3"])


@KINDS
@pytest.mark.parametrize("D,hk,group,page,ctx,drafted,tree,window", [
    (64, 1, 1, 16, [0], [1], "chain", 0),                     # a single key
    (128, 2, 4, 16, [1, 0, 17], [1, 1, 1], "chain", 0),       # single tokens
    (256, 1, 4, 16, [300], [1], "chain", 0),
    (256, 1, 4, 32, [511, 64, 0, 1], [5, 5, 3, 16], "tree", 0),
    (128, 2, 8, 64, [700, 0, 63], [9, 64, 1], "tree", 0),
    (64, 3, 2, 128, [129, 640], [33, 7], "tree", 100),
    (128, 1, 1, 256, [1000], [130], "chain", 0),              # a chunk longer than one tile of rows
    (128, 1, 3, 16, [90], [257], "chain", 64),                # a window inside the chunk
    (64, 2, 5, 32, [257, 31, 200], [70, 1, 66], "tree", 0),   # masks of two words, an odd group
    (128, 4, 2, 16, [1500], [2], "chain", 512),
    (256, 2, 8, 16, [40, 200], [20, 31], "sparse", 0),
    (128, 1, 16, 64, [2049], [64], "tree", 0),
])
def test_attention_matches_oracle(kind, D, hk, group, page, ctx, drafted, tree, window):
    c = Case(D + sum(drafted), kind, D, hk, group, page, ctx, drafted, tree, window)
    c.check(*c.run())


@KINDS
def test_attention_rows_that_see_nothing(kind):
    """No context and a mask that leaves some rows empty: zeros and -inf; a window of one leaves single tokens
    only themselves."""
    c = Case(1, kind, 64, 1, 2, 16, [0, 0], [6, 3], "sparse")
    out, lse = c.run()
    c.check(out, lse)
    assert bool((lse[0] == -float("inf")).all()) and not out[0].any()
    d = Case(2, kind, 128, 1, 1, 16, [50], [1], "chain", window=1)
    d.check(*d.run())


@KINDS
def test_attention_many_splits_and_order(kind):
    """One long sequence on one head (its keys are shared out over the GPU), and the same call twice: equal bits."""
    c = Case(3, kind, 128, 1, 4, 64, [30011], [3], "chain")
    out, lse = c.run()
    c.check(out, lse)
    again = c.run()
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@KINDS
def test_attention_many_sequences(kind):
    """More sequences than SMs, of very different lengths."""
    r = np.random.RandomState(6)
    ctx = [int(x) for x in r.randint(0, 90, 400)]
    ctx[7], ctx[390] = 5000, 3000
    T = [int(x) for x in r.randint(1, 5, 400)]
    c = Case(4, kind, 64, 1, 2, 16, ctx, T, "tree")
    c.check(*c.run())


@KINDS
def test_attention_masked_infinities(kind):
    """A drafted token whose key and value hold infinities and NaN reaches the rows that see it and no other;
    context before the window the same."""
    c = Case(5, kind, 128, 1, 2, 16, [40], [8], "tree", window=24)
    bad = 40 + 3
    k = torch.zeros(2, 1, 128, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 0], k[1] = float("nan"), float("inf")
    aq.aq_kv_write(c.cache, k, k, c.slots[[bad, 2]])
    out, lse = c.run()
    see = [i for i in range(8) if c.bits[0][i, 3]]
    assert see and len(see) < 8
    for i in range(8):
        # position of row i is 40 + depth: key 2 lies before its window
        assert bool(torch.isnan(lse[i]).all()) == (i in see), i
    c.check(out, lse, rows=[i for i in range(8) if i not in see])
    # a value alone: +inf in one element reaches that element of the rows that see it, the others are as before
    if kind == "bf16":
        c = Case(5, kind, 128, 1, 2, 16, [40], [8], "tree", window=24)
        clean, _ = c.run()
        page, off = divmod(int(c.slots[bad]), 16)
        c.cache.v[page, 0, off, 9] = float("inf")
        out, _ = c.run()
        for i in range(8):
            want = clean[i].clone()
            if i in see:
                want[:, 9] = float("inf")
            assert torch.equal(out[i], want), i


@KINDS
def test_attention_scores_of_minus_infinity_and_negative_scale(kind):
    """Keys of minus infinity under positive queries (bf16; an E4M3 cache reads such a key as NaN): rows of zeros
    where no other key is seen, no weight where one is. A negative scale turns the order of the weights round."""
    c = Case(15, kind, 64, 1, 1, 16, [100], [2], "chain")
    if kind == "bf16":
        c.q = c.q.abs() + 0.5
        clean, _ = c.run()
        c.cache.k[..., 0] = torch.where(torch.isnan(c.cache.k[..., 0]), c.cache.k[..., 0], -float("inf"))
        out, lse = c.run()
        assert not out.any() and bool((lse == -float("inf")).all())
        page, off = divmod(int(c.slots[70]), 16)
        c.cache.k[page, 0, off, 0] = 1.0
        out, lse = c.run()
        assert torch.equal(out, c.cache.v[page, 0, off].expand(2, 1, 64)) and bool(torch.isfinite(lse).all())
    d = Case(16, kind, 128, 2, 2, 32, [70], [3], "tree")
    flipped = aq.aq_tree_attention(d.cache, d.q, d.cu, d.ctx_t, d.table, max_q=3, mask=d.mask, depth=d.depth_t, scale=-128 ** -0.5)
    d.q = -d.q
    assert torch.equal(d.run()[0], flipped)


@KINDS
def test_attention_values_of_masked_keys_set_no_scale(kind):
    """A drafted token with values of 1e30 leaves the rows that do not see it as they were."""
    c = Case(17, kind, 128, 1, 2, 16, [40], [8], "tree")
    clean, _ = c.run()
    x = torch.full((1, 1, 128), 1e30, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros_like(x)
    aq.aq_kv_write(c.cache, k, x, c.slots[43:44])
    out, lse = c.run()
    for i in range(8):
        if c.bits[0][i, 3]:
            assert bool((out[i].float().abs() > 1e20).all())
        else:
            assert torch.equal(out[i], clean[i]), i
    c.check(out, lse)


@KINDS
def test_attention_left_out_pages_and_rows(kind):
    """Pages outside the cache and past the table are not read; rows past max_q are not written."""
    c = Case(7, kind, 64, 2, 2, 16, [100], [4], "chain")
    c.table_np[0, 2], c.table_np[0, 4] = -1, 1 << 30
    c.table = torch.from_numpy(c.table_np).cuda()
    c.check(*c.run())
    c.table_np[0, 3:] = -1
    c.table = torch.from_numpy(c.table_np).cuda()[:, :3].contiguous()
    c.check(*c.run())
    c.max_q = 2
    out = torch.full_like(c.q, 5.0)
    aq.aq_tree_attention(c.cache, c.q, c.cu, c.ctx_t, c.table, max_q=2, out=out)
    assert bool((out[2:] == 5).all()) and not bool((out[:2] == 5).all())


@KINDS
def test_attention_strides_streams_workspace(kind):
    c = Case(9, kind, 128, 2, 4, 32, [333, 40], [5, 2], "tree")
    want, lse = c.run()
    wide = torch.full((7, 8 * 128 + 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 256:256 + 1024] = c.q.flatten(1)
    q = wide[:, 256:256 + 1024].unflatten(1, (8, 128))
    out = torch.full((8, 7, 128), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = aq.aq_tree_attention(c.cache, q, c.cu, c.ctx_t, c.table, max_q=5, mask=c.mask, depth=c.depth_t, out=out,
                               stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    # depth left out: the drafted index stands for it, which without a window changes nothing
    assert torch.equal(aq.aq_tree_attention(c.cache, c.q, c.cu, c.ctx_t, c.table, max_q=5, mask=c.mask), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        in_graph, _ = c.run()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(in_graph, want)


@KINDS
def test_attention_extreme_scales(kind):
    """Scores far apart (one key far above the rest), values of very different sizes, and a scale of zero
    (every weight equal)."""
    c = Case(11, kind, 64, 1, 2, 16, [200], [4], "chain", gain=40.0)
    c.check(*c.run())
    for j, g in ((3, 1e4), (90, 1e-4), (150, 0.0)):
        x = (randn(c.r, 1, 1, 64).float() * g).to(torch.bfloat16)
        aq.aq_kv_write(c.cache, randn(c.r, 1, 1, 64), x, c.slots[j:j + 1])
    c.q = randn(c.r, 4, 2, 64)
    c.check(*c.run())
    out = aq.aq_tree_attention(c.cache, c.q, c.cu, c.ctx_t, c.table, max_q=4, scale=0.0)
    V = c.keys()[1]
    for i in range(4):
        mean = V[:200 + i + 1, 0].mean(0)
        tol = 2.0 ** -8 * np.abs(mean) + 1.5 * 2.0 ** -8 * np.abs(V[:200 + i + 1, 0]).mean(0) + 2.0 ** -17 * np.abs(V).max()
        assert np.all(np.abs(f64(out)[i, 0] - mean) <= tol)


def test_attention_offsets_past_32_bits():
    """A cache of more than 2^32 code bytes per array: pages at its far end are read and written."""
    D, hk, page = 128, 8, 256
    pages = (1 << 32) // (D * hk * page) + 8
    cache = aq.KvCache.empty(pages, page, hk, D, aq.AQ_KV_E4M3)
    r = np.random.RandomState(12)
    c = Case(13, "e4m3", D, hk, 1, page, [300], [2], "chain")
    far = [pages - 1, pages - 5]
    slots = torch.tensor([far[j // page] * page + j % page for j in range(302)], dtype=torch.int64, device="cuda")
    k, v = randn(r, 302, hk, D), randn(r, 302, hk, D)
    aq.aq_kv_write(cache, k, v, slots)
    aq.aq_kv_write(c.cache, k, v, c.slots)
    want, lse = c.run()
    c.check(want, lse)
    c.cache, c.table = cache, torch.tensor([far], dtype=torch.int32, device="cuda")
    assert torch.equal(c.run()[0], want)
    got = aq.aq_kv_read(cache, slots)
    code, scale = quantised(v)
    assert torch.equal(got[1], (code * scale[..., None]).to(torch.bfloat16))


# ------------------------------------------------------------------------------------------
# verification
# ------------------------------------------------------------------------------------------
def verify_inputs(seed, sizes, V, shape, with_q):
    """Sequences of `sizes` nodes; probabilities sharpened so that some drafts are accepted."""
    r = np.random.RandomState(seed)
    seqs = []
    for n in sizes:
        logits = 2.0 * r.randn(n + 1, V)
        p = np.exp(logits - logits.max(-1, keepdims=True))
        p = (p / p.sum(-1, keepdims=True)).astype(np.float32)
        logits = logits + 0.8 * r.randn(n + 1, V)
        q = np.exp(logits - logits.max(-1, keepdims=True))
        q = (q / q.sum(-1, keepdims=True)).astype(np.float32)
        if shape == "chain":
            parent = list(range(-1, n - 1))
        elif shape == "wide":
            parent = [-1 if i < 4 else (i - 4) // 3 for i in range(n)]
        else:
            parent = [int(r.randint(-1, i)) if i else -1 for i in range(n)]
        tokens = [int(r.choice(V, p=q[parent[i] + 1].astype(np.float64) / q[parent[i] + 1].sum(dtype=np.float64)))
                  for i in range(n)]
        seqs.append((tokens, parent, p, q if with_q else None, r.rand(n).astype(np.float32),
                     (r.exponential(size=V) + 1e-6).astype(np.float32)))
    return seqs


def run_verify(seqs, shape, dtype=torch.float32, pad=0, cap=None, **kw):
    V = seqs[0][2].shape[1]

    def rows(x):
        t = torch.from_numpy(np.concatenate(x)).to(dtype).cuda()
        if not pad:
            return t
        wide = torch.full((t.size(0), V + pad), float("nan"), dtype=dtype, device="cuda")
        wide[:, :V] = t
        return wide[:, :V]

    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    sizes = [len(s[0]) for s in seqs]
    return aq.aq_verify_drafts(
        rows([s[2] for s in seqs]), i32(sum((s[0] for s in seqs), [])), i32([0] + list(np.cumsum(sizes))),
        torch.from_numpy(np.concatenate([s[4] for s in seqs])).cuda(), torch.from_numpy(np.stack([s[5] for s in seqs])).cuda(),
        q=None if seqs[0][3] is None else rows([s[3] for s in seqs]),
        parent=None if shape == "chain" else i32(sum((s[1] for s in seqs), [])), path_cap=cap, **kw)


VERIFY = [
    (1, [5], 262144, "chain", True), (2, [1, 0, 3], 1000, "chain", True), (3, [7] * 40, 50257, "chain", False),
    (4, [12, 3, 0, 16], 33, "wide", False), (5, [12, 3, 20, 16], 4099, "wide", True), (6, [64, 65, 2], 32000, "random", False),
    (7, [40, 9], 515, "random", True), (8, [6], 1, "chain", True), (9, [300], 8, "random", False), (10, [4] * 700, 64, "wide", True),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("seed,sizes,V,shape,with_q", VERIFY)
def test_verify_matches_oracle(seed, sizes, V, shape, with_q, dtype):
    seqs = verify_inputs(seed, sizes, V, shape, with_q)
    rnd = lambda x: None if x is None else torch.from_numpy(x).to(dtype).double().numpy()  # noqa: E731
    for pad, cap in ((0, None), (3, 2)):
        count, path, token = (t.cpu().numpy() for t in run_verify(seqs, shape, dtype, pad, cap))
        for b, (tokens, parent, p, q, u, noise) in enumerate(seqs):
            want, nxt, margin = serving.verify(tokens, parent, rnd(p), u, noise, q=rnd(q), cap=path.shape[1])
            if margin < 1e-5:     # a comparison that fp32 sums may decide either way
                continue
            assert count[b] == len(want) and path[b].tolist() == want + [-1] * (path.shape[1] - len(want)), (b, margin)
            assert token[b] == nxt, (b, margin)


def test_verify_edges():
    V = 40
    p = np.full((3, V), 1.0 / 32, np.float32)
    p[:, 32:] = 0
    tie = np.ones(V, np.float32)
    # equal scores: the lowest index; a refused token is left out of them
    s = [([0, 1], [-1, -1], p, None, np.array([0.99, 0.99], np.float32), tie)]
    count, path, token = run_verify(s, "tree")
    assert (int(count[0]), path[0].tolist(), int(token[0])) == (0, [-1, -1], 2)
    # u = 0 accepts whatever has mass, and nothing that has none; tokens outside the vocabulary are refused
    s = [([33, V + 5, -3, 7], [-1, -1, -1, -1], np.concatenate([p, p[:2]]), None, np.zeros(4, np.float32), tie)]
    count, path, token = run_verify(s, "tree")
    assert (int(count[0]), path[0].tolist(), int(token[0])) == (1, [3, -1, -1, -1], 0)
    # p equal to q leaves no residual: accepted for every u below one; every token refused: the draw is from p
    one = np.zeros((2, V), np.float32)
    one[:, 9] = 1.0
    s = [([9], [-1], one, one, np.array([1.0], np.float32), tie)]
    assert int(run_verify(s, "chain")[2][0]) == 9
    # no drafts: a plain draw; an empty batch; a parent that points forward is never reached
    s = [([], [], one[:1], None, np.zeros(0, np.float32), tie)]
    count, path, token = run_verify(s, "chain")
    assert (int(count[0]), tuple(path.shape), int(token[0])) == (0, (1, 0), 9)
    s = [([9, 9], [1, -1], np.concatenate([one, one[:1]]), None, np.zeros(2, np.float32), tie)]
    count, path, _ = run_verify(s, "tree")
    assert path[0].tolist() == [1, -1]
    # a repeated sibling has no mass left the second time
    half = np.zeros((3, V), np.float32)
    half[:, 3], half[:, 4] = 0.5, 0.5
    s = [([3, 3], [-1, -1], half, None, np.array([0.6, 0.0], np.float32), tie)]
    count, path, token = run_verify(s, "tree")
    assert int(count[0]) == 0 and int(token[0]) == 4


def test_verify_repeats_and_graph():
    seqs = verify_inputs(21, [6] * 30, 32000, "wide", True)
    a = run_verify(seqs, "wide")
    b = run_verify(seqs, "wide")
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("with_q", [True, False])
def test_verify_padded_trees(with_q, dtype):
    """Trees padded to one shape with nodes that have no token: as the oracle's, and as the trees without them."""
    r = np.random.RandomState(31)
    seqs = verify_inputs(30, [12] * 40, 1000, "wide", with_q)
    for b, s in enumerate(seqs):
        for i in range(12):
            if r.rand() < (1.0 if b < 4 else 0.4):
                s[0][i] = int(r.choice([-1, 1000, -2 ** 31]))
    rnd = lambda x: None if x is None else torch.from_numpy(x).to(dtype).double().numpy()  # noqa: E731
    count, path, token = (t.cpu().numpy() for t in run_verify(seqs, "wide", dtype, cap=12))
    for b, (tokens, parent, p, q, u, noise) in enumerate(seqs):
        want, nxt, margin = serving.verify(tokens, parent, rnd(p), u, noise, q=rnd(q), cap=12)
        if b < 4:
            assert nxt == int((rnd(p)[0] / noise.astype(np.float64)).argmax())
        if margin >= 1e-5:
            assert count[b] == len(want) and path[b].tolist() == want + [-1] * (12 - len(want)) and token[b] == nxt, b


@pytest.mark.parametrize("layout", [aq.AQ_ROPE_HALF, aq.AQ_ROPE_INTERLEAVED], ids=["half", "interleaved"])
@pytest.mark.parametrize("D,rot", [(128, 64), (128, 16), (256, 128), (64, 48), (80, 32)])
def test_rotation_of_a_part_leaves_the_rest(layout, D, rot):
    """What lies past rotary_dim comes through bit for bit: infinities, zeros of either sign, the largest and the smallest."""
    r = np.random.RandomState(D + rot)
    rest = torch.tensor([float("inf"), -0.0, -float("inf"), 0.0, 3e38, -1e-39, 1.0, -1.0])
    x = randn(r, 9, 3, D)
    x[..., rot:] = rest.repeat((D - rot + 7) // 8)[:D - rot].to(torch.bfloat16).cuda()
    rope = aq.rope_frequencies(rot, layout=layout)
    pos = torch.tensor([0, 1, 5, 100, 7, 8, 9, 1000, -3], dtype=torch.int32, device="cuda")
    bits = lambda t: t.contiguous().view(torch.int16)  # noqa: E731
    for inverse in (False, True):
        y = aq.aq_rope(rope, pos, x, inverse=inverse)
        assert torch.equal(bits(y[..., rot:]), bits(x[..., rot:]))
        rope_ok(f64(y[..., :rot]), f64(x[..., :rot]), pos.cpu().numpy(), *serving.rope_angles(rot),
                "half" if layout == aq.AQ_ROPE_HALF else "interleaved", inverse=inverse)
    if D in (64, 128, 256):
        cache = aq.KvCache.empty(2, 16, 3, D, aq.AQ_KV_BF16)
        slots = torch.arange(9, device="cuda")
        q = aq.aq_kv_write(cache, x, x, slots, rope=rope, pos=pos, q=x)
        k, v = aq.aq_kv_read(cache, slots)
        assert torch.equal(bits(q[..., rot:]), bits(x[..., rot:])) and torch.equal(bits(k[..., rot:]), bits(x[..., rot:]))
        assert torch.equal(bits(v), bits(x))


def test_rotation_records_no_history_and_its_inverse_is_the_backward_pass():
    """As the call's documentation says: used in a step of torch's own by a function whose backward pass is the inverse call."""
    r = np.random.RandomState(40)
    x, g = randn(r, 6, 2, 64).requires_grad_(), randn(r, 6, 2, 64)
    rope, pos = aq.rope_frequencies(64), torch.arange(6, dtype=torch.int32, device="cuda") * 50
    assert not aq.aq_rope(rope, pos, x).requires_grad

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return aq.aq_rope(rope, pos, x)

        @staticmethod
        def backward(ctx, g):
            return aq.aq_rope(rope, pos, g, inverse=True)

    Turn.apply(x).backward(g)
    rope_ok(f64(x.grad), f64(g), pos.cpu().numpy(), *serving.rope_angles(64), "half", inverse=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_verify_draws_among_subnormal_probabilities(dtype):
    """Rows whose probabilities, or whose noise, lie below the normal numbers: the largest quotient, the lowest of equal ones."""
    r = np.random.RandomState(50)
    B, V = 64, 5000
    unit = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133
    p = torch.from_numpy((r.randint(0, 12, (B, V)) * unit).astype(np.float32)).to(dtype).cuda()
    p[1::2] = torch.from_numpy(r.rand(B // 2, V).astype(np.float32)).to(dtype).cuda()
    noise = (r.exponential(size=(B, V)) + 1e-6).astype(np.float32)
    noise[1::2] = (r.randint(1, 50, (B // 2, V)) * 2.0 ** -149).astype(np.float32)
    p[1::2] *= 2.0 ** -30    # quotients that fp32 holds
    empty, none = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda")
    _, _, token = aq.aq_verify_drafts(p, empty, torch.zeros(B + 1, dtype=torch.int32, device="cuda"), none, torch.from_numpy(noise).cuda())
    score = (p.double().cpu().numpy() / noise.astype(np.float64)).astype(np.float32)      # to fp32 as the kernel divides
    assert np.array_equal(token.cpu().numpy(), score.argmax(1))
