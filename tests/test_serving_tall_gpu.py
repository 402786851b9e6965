"""Attention over tall row tiles (more than 32 rows of a key/value head, the tcgen05 kernel) at special values, with several key
tiles; and the bounds that include/aq.h states for an E4M3 cache, in both kernels. Tolerances: those of test_serving_items_gpu.
"""
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from test_serving_items_gpu import Batch, KINDS, no_wait_ran_out  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# one row tile, two row tiles, D = 256
TALL = pytest.mark.parametrize("D,T", [(64, 24), (64, 64), (128, 24), (128, 64), (256, 64)])


def rows_that_see(c, b, j):
    """Rows (over all sequences) of sequence b that see its drafted token j."""
    return [int(c.cu_np[b]) + i for i in range(c.T[b]) if c.bits[b][i, j]]


def put(c, b, j, k=None, v=None):
    """Key j (of context and drafted tokens) of sequence b takes these keys or values; nothing else changes."""
    at = int(c.first[b]) + j
    if k is not None:
        c.k[at] = k
    if v is not None:
        c.v[at] = v
    aq.aq_kv_write(c.cache, c.k[at:at + 1], c.v[at:at + 1], c.slots[at:at + 1])


@KINDS
@TALL
def test_masked_infinities(kind, D, T):
    """A drafted token of infinities and NaN in key and value reaches the rows that see it, and no other."""
    c = Batch(D + T, kind, D, 2, 4, 16, [300, 7], [T, T], tree=True)
    put(c, 0, 300 + 3, k=float("nan"), v=float("inf"))
    put(c, 1, 7 + 5, k=float("inf"), v=float("nan"))
    see = rows_that_see(c, 0, 3) + rows_that_see(c, 1, 5)
    assert 2 < len(see) < 2 * T
    out, lse = c.run()
    for i in see:
        assert bool(torch.isnan(lse[i]).all()) and bool(torch.isnan(out[i]).all()), i
    # the others: as though the token held zeros
    for b, j in ((0, 303), (1, 12)):
        put(c, b, j, k=0.0, v=0.0)
    c.check(out, lse, skip=see)


@KINDS
@pytest.mark.parametrize("where", ["drafted", "context"])
@pytest.mark.parametrize("D,T", [(64, 24), (64, 64), (128, 24), (128, 64), (256, 64), (128, 2), (64, 4), (256, 8)])
def test_a_value_alone(kind, D, T, where):
    """An infinite value (with an E4M3 cache: a vector that reads as NaN) under a finite key: the rows that see it have it in
    their output, their lse and every other row are as with a finite value there."""
    c = Batch(D + T + 1, kind, D, 2, 4, 32, [400], [T], tree=True)
    key = 401 if where == "drafted" else 130
    see = rows_that_see(c, 0, 1) if where == "drafted" else range(T)
    at = int(c.first[0]) + key
    v, finite = c.v[at].clone(), c.v[at].clone()
    v[:, 9] = float("inf")
    put(c, 0, key, v=v)
    out, lse = c.run()
    for i in see:
        if kind == "bf16":
            assert bool((out[i, :, 9] == float("inf")).all()) and bool(torch.isfinite(out[i, :, 10:]).all()), i
        else:
            assert bool(torch.isnan(out[i]).all()), i
    put(c, 0, key, v=finite)
    c.check(out, lse, skip=see)
    want, want_lse = c.run()
    assert float((lse - want_lse).abs().max()) < 2e-5 + 1e-6 * float(want_lse.abs().max())


@KINDS
@TALL
def test_values_of_masked_keys_set_no_scale(kind, D, T):
    c = Batch(D + T + 2, kind, D, 1, 4, 16, [150], [T], tree=True)
    put(c, 0, 150 + 4, k=0.0, v=1e30)
    see = rows_that_see(c, 0, 4)
    out, lse = c.run()
    c.check(out, lse)
    for i in see:
        assert bool((out[i].float().abs() > 1e20).all())


@KINDS
@TALL
def test_scores_that_grow_and_values_of_all_sizes(kind, D, T):
    """Every tile passes the reference of the one before; later the values' sizes do."""
    c = Batch(D + T + 3, kind, D, 2, 4, 64, [700, 90], [T, T - 3], tree=True)
    n = int(c.first[1])
    step = torch.arange(n, device="cuda")[:, None, None] / n
    c.k[:n] = (c.k[:n].float() * (0.2 + 6 * step)).to(torch.bfloat16)
    c.write()
    c.check(*c.run())
    c.v[:n] = (c.v[:n].float() * torch.exp2(torch.round(40 * step - 20))).to(torch.bfloat16)
    c.write()
    c.check(*c.run())
    c.v[:n] = c.v[:n].flip(0).clone()
    c.write()
    c.check(*c.run())


@KINDS
@TALL
def test_scale_zero_and_negative_scale(kind, D, T):
    c = Batch(D + T + 4, kind, D, 1, 4, 16, [260], [T], tree=True)
    out = aq.aq_tree_attention(c.cache, c.q, c.cu, c.ctx_t, c.table, max_q=c.max_q, mask=c.mask, depth=c.depth, scale=0.0)
    q, c.q = c.q, torch.zeros_like(c.q)
    want, lse = c.run()
    c.check(want, lse)
    c.check(out, lse)
    c.q = q
    flipped = aq.aq_tree_attention(c.cache, c.q, c.cu, c.ctx_t, c.table, max_q=c.max_q, mask=c.mask, depth=c.depth, scale=-D ** -0.5)
    c.q = -c.q
    assert torch.equal(c.run()[0], flipped)


@TALL
def test_scores_of_minus_infinity(D, T):
    """Keys of minus infinity under positive queries: zeros and lse -inf where no other key is seen; one finite key is all."""
    c = Batch(D + T + 5, "bf16", D, 1, 4, 16, [300], [T])
    c.q = c.q.abs() + 0.5
    c.k[:, :, 0] = -float("inf")
    c.write()
    out, lse = c.run()
    assert not bool(out.any()) and bool((lse == -float("inf")).all())
    put(c, 0, 170, k=1.0)
    out, lse = c.run()
    assert bool(torch.isfinite(lse).all()) and torch.equal(out, c.v[170, 0].expand_as(out))


@KINDS
@TALL
def test_left_out_pages_and_empty_rows(kind, D, T):
    """A page the table does not name, and trees whose even rows see nothing of a sequence without context."""
    c = Batch(D + T + 6, kind, D, 2, 4, 16, [0, 130], [T, T], tree=True)
    mask = c.mask.clone()
    for i in range(0, T, 2):
        mask[i] = 0
        c.bits[0][i] = False
    c.mask = mask
    out, lse = c.run()
    c.check(out, lse)
    assert bool((lse[0:T:2] == -float("inf")).all()) and not bool(out[0:T:2].any())
    full, _ = c.run()
    c.table[1, 2] = -1
    gone, lse = c.run()
    see = c.seen(1)
    c.seen = lambda b: see if b == 1 else Batch.seen(c, b)
    see[:, 32:48] = False
    c.check(gone, lse)
    assert not torch.equal(gone[T:], full[T:])


@pytest.mark.parametrize("D,T,group", [(64, 1, 4), (128, 2, 4), (128, 8, 4), (256, 8, 4), (64, 24, 4), (128, 64, 4), (256, 64, 2), (128, 30, 2)])
def test_e4m3_queries_keep_elements_far_below_the_largest(D, T, group):
    """One element of 1024 meets keys of zero there; the scores come from the elements 2^-18 to 2^-25 below it. (Held in fewer
    bits or with less range they would be lost: every weight equal.)"""
    c = Batch(D + T + 7, "e4m3", D, 1, group, 16, [90], [T], tree=True)
    c.k = (c.k.float() * 2.0 ** 12).to(torch.bfloat16)
    c.k[:, :, 0] = 0
    c.write()
    c.q = (torch.randn(*c.q.shape, generator=c.g, device="cuda") * 2.0 ** -11).to(torch.bfloat16)
    c.q[:, :, 0] = 1024.0
    out, lse = c.run()
    c.check(out, lse)
    c.q[:, :, 1:] = 0
    assert float((c.run()[1] - lse).abs().min()) > 1e-3


@pytest.mark.parametrize("D,T,group", [(64, 1, 1), (128, 2, 4), (128, 8, 4), (256, 8, 4), (64, 24, 4), (128, 64, 4), (256, 64, 2)])
def test_e4m3_weights_have_eleven_bits(D, T, group):
    """Two keys whose values nearly cancel: what is left shows the weights' own rounding, 2^-11 of a, and not bf16's 2^-8."""
    c = Batch(D + T + 8, "e4m3", D, 1, group, 16, [2], [T], tree=True)
    for i in range(T):     # every row sees the two context tokens alone
        c.bits[0][i] = False
    c.mask = torch.zeros_like(c.mask)
    c.q = (c.q.float() * 0.5).to(torch.bfloat16)
    c.v[0], c.v[1] = 448.0, -448.0
    r = torch.randint(0, 8, (D,), generator=c.g, device="cuda")
    c.v[1, 0] = -(torch.tensor([448.0, 416, 384, 352, 320, 288, 256, 240], device="cuda")[r]).to(torch.bfloat16)
    c.v[1, 0, 0], c.v[0, 0, 1:] = -448.0, torch.tensor([448.0, 416, 384, 352, 320, 288, 256, 240], device="cuda")[r.flip(0)][1:].to(torch.bfloat16)
    c.write()
    c.check(*c.run())


@pytest.mark.parametrize("spread", [12, 40])
@pytest.mark.parametrize("D,T,group", [(64, 1, 4), (128, 1, 4), (128, 8, 4), (256, 8, 4), (64, 24, 4), (64, 64, 4), (128, 24, 4), (128, 64, 4), (256, 64, 2)])
def test_e4m3_large_logits_on_keys_of_small_values(D, T, group, spread):
    """Context in which every other key has the larger logit, by about `spread` powers of two, and values smaller by as many: no
    key's weight times scale is far from another's, and none may be lost for the largest logit's and the largest scale's sake."""
    c = Batch(D + T + 9, "e4m3", D, 1, group, 32, [700], [T], tree=True)
    c.q = (c.q.float() * 0.25).to(torch.bfloat16)
    c.q[:, :, 0] = 4.0
    up = (torch.arange(c.k.size(0), device="cuda") % 2 == 0)[:, None]
    c.k[:, :, 0] = torch.where(up, spread * 0.6931 * D ** 0.5 / 8.0, -spread * 0.6931 * D ** 0.5 / 8.0).to(torch.bfloat16)
    c.v = (c.v.float() * torch.where(up, 2.0 ** -spread, 1.0)[..., None]).to(torch.bfloat16)
    c.write()
    c.check(*c.run())
    # the same with the small values under the small logits: those are dropped, within the bound
    c.v = c.v.roll(1, 0)
    c.write()
    c.check(*c.run())
