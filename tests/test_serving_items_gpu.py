"""Attention in which one CTA walks from item to item, against the formulas in float64 on the GPU.

The calls here hold more items than CTAs, or more key tiles than the short-call rule takes, so that query buffers, score
buffers and sums are used again by the next item while other warps are still at the last one; sequences of one token stand
beside full ones, so that some warps have no row and run ahead.

Tolerances, from the formats that include/aq.h states (unit roundoffs: bf16 2^-8, f16 2^-11, fp32 2^-24; n keys seen, p the
weights, a = sum p |v|):
  output      its bf16 rounding: 2^-8 |o|
  weights     bf16 cache: 2^-8 of each, 2^-8 a, and half as much for the exponential and the sums.
              E4M3 cache: 2^-11 of each, 2^-11 a; below 2^-22 of the row's largest weight times scale, half a step of f16's
              smallest: n 2^-33 of that largest, for codes of up to 448; 2^-16 a for the exponential, n 2^-25 a for the fp32 sums
  scores      fp32 sums of D products, 2^-20 of sum |q||k|; E4M3: query elements below 2^-28 of the largest lost; a weight is
              off by twice a score's error
  lse         a score's error, the exponential and logarithm (2e-5), its fp32 rounding
"""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq

pytestmark = pytest.mark.gpu

DT = {"bf16": aq.AQ_KV_BF16, "e4m3": aq.AQ_KV_E4M3}
KINDS = pytest.mark.parametrize("kind", ["bf16", "e4m3"])


@pytest.fixture(autouse=True)
def no_wait_ran_out():
    yield
    assert aq.aq_device_status() == aq.AQ_OK


class Batch:
    """Sequences of ctx context and drafted tokens in a paged cache whose every unnamed cell is NaN."""

    def __init__(self, seed, kind, D, hk, group, page, ctx, drafted, tree=False, window=0, gain=1.0):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.RandomState(seed)
        self.kind, self.D, self.hk, self.group, self.page, self.window = kind, D, hk, group, page, window
        self.ctx, self.T = list(ctx), list(drafted)
        need = [-(-(c + t) // page) for c, t in zip(self.ctx, self.T)]
        pages = sum(need) + 2
        order = r.permutation(pages)[:sum(need)].astype(np.int32)
        table = np.full((len(need), max(need)), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.cache = aq.KvCache.empty(pages, page, hk, D, DT[kind])
        for t in (self.cache.k, self.cache.v):
            t.fill_(0x7f if kind == "e4m3" else float("nan"))
        if kind == "e4m3":
            self.cache.k_scale.fill_(float("nan"))
            self.cache.v_scale.fill_(float("nan"))
        self.first = np.concatenate([[0], np.cumsum([c + t for c, t in zip(self.ctx, self.T)])])
        self.slots = torch.from_numpy(np.concatenate(
            [table[b, np.arange(c + t) // page].astype(np.int64) * page + np.arange(c + t) % page
             for b, (c, t) in enumerate(zip(self.ctx, self.T))])).cuda()
        n, total = int(self.first[-1]), sum(self.T)
        self.k, self.v = self.randn(n, hk, D), self.randn(n, hk, D)
        self.write()
        self.q = (self.randn(total, hk * group, D).float() * gain).to(torch.bfloat16)
        self.cu_np = np.concatenate([[0], np.cumsum(self.T)])
        self.cu = torch.from_numpy(self.cu_np.astype(np.int32)).cuda()
        self.ctx_t = torch.tensor(self.ctx, dtype=torch.int32, device="cuda")
        self.max_q = max(self.T)
        self.mask = self.depth = self.bits = None
        if tree:
            words = -(-self.max_q // 64)
            m, depth, self.bits = np.zeros((total, words), np.uint64), np.zeros(total, np.int32), []
            for b, t in enumerate(self.T):
                bits = np.zeros((t, t), bool)
                for i in range(t):
                    par = r.randint(max(-1, i - 9), i) if i else -1
                    if par >= 0:
                        bits[i] = bits[par]
                        depth[self.cu_np[b] + i] = depth[self.cu_np[b] + par] + 1
                    bits[i, i] = True
                self.bits.append(bits)
                for i, j in np.argwhere(bits):
                    m[self.cu_np[b] + i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
            self.mask, self.depth = torch.from_numpy(m.view(np.int64)).cuda(), torch.from_numpy(depth).cuda()

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def write(self):
        aq.aq_kv_write(self.cache, self.k, self.v, self.slots)

    def run(self, **kw):
        return aq.aq_tree_attention(self.cache, self.q, self.cu, self.ctx_t, self.table, max_q=self.max_q, mask=self.mask,
                                    depth=self.depth, window=self.window, return_lse=True, **kw)

    def stored(self):
        """k, v [keys, heads, D] as the cache holds them, in float64, and the values' scales."""
        got = []
        for codes, scale in ((self.cache.k, self.cache.k_scale), (self.cache.v, self.cache.v_scale)):
            flat = codes.transpose(1, 2).reshape(-1, self.hk, self.D)[self.slots]
            s = torch.ones(flat.shape[:2], dtype=torch.float64, device="cuda")
            if scale is not None:
                flat, s = flat.view(torch.float8_e4m3fn), scale.transpose(1, 2).reshape(-1, self.hk)[self.slots].double()
            got.append((flat.double() * s[..., None], s))
        return got[0][0], got[1][0], got[1][1]

    def seen(self, b):
        c, t = self.ctx[b], self.T[b]
        i = torch.arange(t, device="cuda")
        see = torch.ones(t, c + t, dtype=torch.bool, device="cuda")
        if self.bits is None:
            depth, see[:, c:] = i, i[:, None] >= i[None]
        else:
            depth = self.depth[self.cu_np[b]:self.cu_np[b + 1]].long()
            see[:, c:] = torch.from_numpy(self.bits[b]).cuda()
        if self.window > 0:
            where = torch.cat([torch.arange(c, device="cuda"), c + depth])
            see &= (c + depth)[:, None] - where[None] < self.window
        return see

    def check(self, out, lse, skip=()):
        """Every row of every sequence (but rows `skip`, counted over all) within the tolerance."""
        K, V, S = self.stored()
        worst = 0.0
        for b, (c, t) in enumerate(zip(self.ctx, self.T)):
            if t == 0:
                continue
            at = slice(int(self.first[b]), int(self.first[b + 1]))
            see = self.seen(b)
            # [heads, t, group, ...]
            q = self.q[self.cu_np[b]:self.cu_np[b + 1]].double().view(t, self.hk, self.group, self.D).permute(1, 0, 2, 3)
            k, v, s = K[at].transpose(0, 1), V[at].transpose(0, 1), S[at].transpose(0, 1)
            # cells that no row sees may hold anything
            none = ~see.any(0)
            k, v, s = (x.masked_fill(none[None, :, None] if x.dim() == 3 else none[None], 0.0) for x in (k, v, s))
            scale = self.D ** -0.5
            x = torch.einsum("htgd,hkd->htgk", q, k) * scale
            x = x.masked_fill(~see[None, :, None], -float("inf"))
            want_lse = torch.logsumexp(x, -1)
            p = torch.nan_to_num(torch.exp(x - want_lse[..., None]))
            o, a = torch.einsum("htgk,hkd->htgd", p, v), torch.einsum("htgk,hkd->htgd", p, v.abs())
            n = see.sum(-1).double()[None, :, None]
            e = 2.0 ** -20 * torch.einsum("htgd,hkd->htgk", q.abs(), k.abs()).masked_fill(~see[None, :, None], 0).amax(-1)
            if self.kind == "e4m3":
                e = e + 2.0 ** -28 * q.abs().amax(-1) * (k.abs().sum(-1)[:, None, None] * see[None, :, None]).amax(-1)
                low = n * 2.0 ** -33 * 448.0 * (p * s[:, None, None]).amax(-1)
                rel = 2.0 ** -11 + 2.0 ** -16 + n * 2.0 ** -25
            else:
                low, rel = torch.zeros_like(e), torch.full_like(e, 1.5 * 2.0 ** -8)
            e = e * scale
            tol = 2.0 ** -8 * o.abs() + (rel + 4 * e)[..., None] * a + low[..., None]
            got = out[self.cu_np[b]:self.cu_np[b + 1]].double().view(t, self.hk, self.group, self.D).permute(1, 0, 2, 3)
            got_lse = lse[self.cu_np[b]:self.cu_np[b + 1]].double().view(t, self.hk, self.group).permute(1, 0, 2)
            bad = ~((got - o).abs() <= tol)
            bad_lse = ~((got_lse - want_lse).abs() <= e + 2e-5 + 1e-6 * want_lse.abs()) & ~((got_lse == want_lse) & (want_lse == -float("inf")))
            for i in range(t):
                if int(self.cu_np[b]) + i in skip:
                    bad[:, i], bad_lse[:, i] = False, False
            assert not bool(bad.any()), (b, c, t, torch.nonzero(bad)[:3].tolist(), float((got - o).abs()[bad].max()), float(tol[bad].min()))
            assert not bool(bad_lse.any()), (b, c, t, torch.nonzero(bad_lse)[:3].tolist())
            worst = max(worst, float(((got - o).abs() / tol.clamp_min(1e-300)).nan_to_num(0.0).max()))
        return worst


DIMS = pytest.mark.parametrize("D", [64, 128, 256])


@KINDS
@DIMS
@pytest.mark.parametrize("group,T", [(2, [1, 64]), (2, [64, 1, 33, 2, 17, 64]), (4, [1, 64, 33, 2]), (3, [43, 1, 42])],
                         ids=["one-full", "mixed", "two-tiles", "odd-group"])
def test_many_items_of_different_heights(kind, D, group, T):
    """Hundreds of items, short ones beside full ones: 2 to 128 rows of a tile of 128, 4 to 256 of 256."""
    r = np.random.RandomState(D + group)
    drafted = [T[i % len(T)] for i in range(150)]
    c = Batch(D + group, kind, D, 2, group, 32, [int(x) for x in r.randint(0, 500, 150)], drafted)
    c.check(*c.run())


@KINDS
@DIMS
def test_many_items_just_past_a_tile(kind, D):
    """Rows 1 to 3 past a multiple of 128, and the next sequence's full."""
    r = np.random.RandomState(D)
    drafted = [[129, 128, 130, 256, 131, 257, 1][i % 7] for i in range(70)]
    c = Batch(D + 1, kind, D, 3, 1, 64, [int(x) for x in r.randint(0, 300, 70)], drafted)
    c.check(*c.run())


@KINDS
@DIMS
@pytest.mark.parametrize("group", [2, 4])
def test_long_contexts_mixed_with_single_tokens(kind, D, group):
    """Few items of many tiles each: more than six key tiles a CTA, cut anywhere, single tokens beside trees of 64."""
    drafted = [1, 64] * 8
    c = Batch(D + group, kind, D, 2, group, 64, [9000 - 137 * i for i in range(16)], drafted, tree=True)
    c.check(*c.run())


@KINDS
@DIMS
def test_window_and_trees_over_many_items(kind, D):
    r = np.random.RandomState(D + 5)
    drafted = [int(x) for x in r.randint(1, 130, 120)]
    c = Batch(D + 5, kind, D, 2, 2, 16, [int(x) for x in r.randint(0, 900, 120)], drafted, tree=True, window=200)
    c.check(*c.run())


@KINDS
def test_max_q_far_above_most_sequences(kind):
    """Row tiles that most sequences do not have."""
    r = np.random.RandomState(2)
    drafted = [1 + i % 3 for i in range(200)]
    drafted[50] = 700
    c = Batch(3, kind, 128, 2, 2, 32, [int(x) for x in r.randint(0, 700, 200)], drafted)
    c.check(*c.run())


@KINDS
@DIMS
@pytest.mark.parametrize("group", [2, 4])
def test_items_repeat_bit_for_bit(kind, D, group):
    """Equal calls give equal bits, however the warps of a CTA run ahead of one another and whatever shared memory held before:
    row tiles of which some are partly filled, other calls in between."""
    r = np.random.RandomState(4)
    drafted = [[1, 64, 33][i % 3] for i in range(160)]
    c = Batch(D + 7, kind, D, 2, group, 32, [int(x) for x in r.randint(0, 800, 160)], drafted)
    d = Batch(D + 8, kind, D, 1, 2 * group, 32, [int(x) for x in r.randint(0, 300, 40)], [64] * 40, gain=30.0)
    out, lse = c.run()
    for _ in range(20):
        again = c.run()
        d.run()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@KINDS
@DIMS
@pytest.mark.parametrize("T", [[0, 64, 1, 0, 0, 33], [0, 1, 3, 0], [0, 0, 0, 5]], ids=["tall", "short", "few"])
def test_sequences_without_rows_between_others(kind, D, T):
    r = np.random.RandomState(D + 9)
    drafted = [T[i % len(T)] for i in range(90)]
    c = Batch(D + 9, kind, D, 2, 2, 16, [int(x) for x in r.randint(0, 400, 90)], drafted, tree=True)
    c.check(*c.run())


@KINDS
@DIMS
@pytest.mark.parametrize("T", [1, 3, 6, 9])
def test_short_items_repeat_bit_for_bit(kind, D, T):
    """The same for row tiles of 8, 16 and 32, with tall calls in between."""
    r = np.random.RandomState(T)
    c = Batch(D + T, kind, D, 2, 4, 32, [int(x) for x in r.randint(0, 700, 170)], [1 + i % T for i in range(170)])
    d = Batch(D + 8, kind, D, 1, 4, 32, [int(x) for x in r.randint(0, 300, 40)], [40] * 40, gain=30.0)
    out, lse = c.run()
    c.check(out, lse)
    for _ in range(10):
        d.run()
        again = c.run()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@KINDS
@DIMS
@pytest.mark.parametrize("T", [5, 40, 64])
def test_strided_rows(kind, D, T):
    """Queries as columns of a wider row, outputs with heads outermost or as columns; nothing beside them is written."""
    c = Batch(D + T, kind, D, 2, 4, 32, [500, 3, 77], [T, 1, T - 2], tree=True)
    want, lse = c.run()
    total = c.q.size(0)
    wide = torch.full((total, 10 * D), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, D:9 * D] = c.q.flatten(1)
    c.q = wide[:, D:9 * D].unflatten(1, (8, D))
    heads = torch.full((8, total + 2, D), 7.0, dtype=torch.bfloat16, device="cuda")
    got, _ = c.run(out=heads[:, 1:-1].transpose(0, 1))
    assert torch.equal(got, want) and bool((heads[:, 0] == 7).all()) and bool((heads[:, -1] == 7).all())
    cols = torch.full((total, 10 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(out=cols[:, D:9 * D].unflatten(1, (8, D)))
    assert torch.equal(cols[:, D:9 * D].unflatten(1, (8, D)), want) and bool((cols[:, :D] == 7).all()) and bool((cols[:, 9 * D:] == 7).all())
