"""Token scores and their gradient on the GPU against the float64 oracle.

Tolerances. Words that hold more than 2^-24 of a row lie within 30 of its largest z, for rows of up to 2^18 words. Their exponents are
off by 2^-23 of that (a difference and a product), a power of two by 2^-22 of itself, and a sum of n words in chains of at most
min(n, 4096) by that many 2^-24: the logarithm of the sum of e^(z - max), and the sum of p (z - max), by
2^-24 (8 x 30 + 16 + min(n, 4096)); logprob has its own 2^-23 besides, lse its, and entropy that times 1 + H. Words and their order are
exact. The gradient: p's exponent is off by 2^-23 of |log p|, so a term by 2^-20 (1 + |log p|) of itself, and the output's
rounding."""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from oracle import serving

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def logits(r, rows, vocab, dtype, by=3.0):
    return torch.from_numpy((by * r.standard_normal((rows, vocab))).astype(np.float32)).to(DT[dtype]).cuda()


def same(got, ref, tol):
    """Equal where the reference is not finite, within tol elsewhere."""
    ref, tol = np.asarray(ref), np.broadcast_to(tol, np.shape(ref))
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine], equal_nan=True), (got[~fine][:4], ref[~fine][:4])
    d = np.abs(got[fine] - ref[fine])
    assert (d <= tol[fine]).all(), (d.max(), tol[fine].min())


def check(x, tokens, scale, top, **kw):
    r = aq.aq_token_logprobs(x, tokens, scale=scale, top=top, **kw)
    X = f64(x)
    lp, lse, h, tl, tt = serving.token_scores(X, None if tokens is None else tokens.cpu().numpy(), np.float64(np.float32(scale)), top)
    tol = 2.0 ** -24 * (8 * 30 + 16 + min(X.shape[1], 4096))
    size = lambda v: np.abs(np.nan_to_num(v, posinf=0, neginf=0))  # noqa: E731
    same(f64(r.lse), lse, tol + 2.0 ** -23 * size(lse))
    same(f64(r.entropy), h, tol * (1 + size(h)))
    if tokens is not None:
        same(f64(r.logprob), lp, tol + 2.0 ** -23 * size(lp))
    else:
        assert r.logprob is None
    if top:
        assert np.array_equal(r.top_token.cpu().numpy(), tt)
        same(f64(r.top_logprob), tl, tol + 2.0 ** -23 * size(tl))
    else:
        assert r.top_token is None and r.top_logprob is None
    return r


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,top,scale", [
    (1, 1, 1, 1.0), (3, 2, 2, 1.0), (2, 7, 5, 0.5), (4, 31, 31, 1.0), (5, 33, 32, 2.0), (1, 1000, 20, 1.0), (7, 1025, 32, 1.25),
    (3, 8191, 3, 1.0), (200, 4097, 20, 0.7), (2, 32003, 20, 1.0), (40, 50257, 5, 1.0), (1, 262144, 32, 1.0), (5, 262144, 5, 1.0),
    (1000, 300, 1, 1.0), (700, 5000, 0, 1.0), (12, 151936, 1, 0.9),
])
def test_scores(rows, vocab, top, scale, dtype):
    r = np.random.RandomState(rows + vocab)
    x = logits(r, rows, vocab, dtype)
    tokens = torch.from_numpy(r.randint(0, vocab, rows).astype(np.int32)).cuda()
    if rows > 2:
        tokens[1], tokens[2] = -1, vocab
    a = check(x, tokens, scale, top)
    b = aq.aq_token_logprobs(x, tokens, scale=scale, top=top)
    assert all(u is v is None or torch.equal(u, v) for u, v in zip(a, b))     # the sums' order is fixed
    check(x, None, scale, top)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [9, 3000, 70000])
@pytest.mark.parametrize("shape", ["constant", "rising", "falling", "two values", "mostly -inf", "all -inf", "lowest", "nan", "inf", "zeros", "steps"])
def test_rows_that_are_hard(shape, vocab, dtype):
    """Ties everywhere, orders that renew the list at every word, masks by -inf and by the type's lowest value, NaN, infinities."""
    r = np.random.RandomState(vocab)
    x = np.zeros((3, vocab), np.float32)
    i = np.arange(vocab, dtype=np.float32)
    if shape == "constant":
        x[:] = 2.5
    elif shape == "rising":
        x[:] = i / vocab * 20
    elif shape == "falling":
        x[:] = -i / vocab * 20
    elif shape == "two values":
        x[:] = r.randint(0, 2, x.shape)
    elif shape == "mostly -inf":
        x[:] = -np.inf
        x[0, vocab // 2], x[1, [0, vocab - 1]], x[2, 3:6] = 1.0, -3.0, 7.0
    elif shape == "all -inf":
        x[:] = -np.inf
    elif shape == "lowest":
        x[:] = torch.finfo(DT[dtype]).min
        x[0, vocab - 2], x[1, 1] = 0.0, 5.0
    elif shape == "nan":
        x[:] = r.standard_normal(x.shape)
        x[0, vocab // 3], x[1, :] = np.nan, np.nan
        x[2, 0], x[2, -1] = -np.inf, np.nan
    elif shape == "inf":
        x[:] = r.standard_normal(x.shape)
        x[0, vocab // 3], x[1, [1, vocab - 1]] = np.inf, np.inf
        x[2, 2], x[2, 5] = np.inf, -np.inf
    elif shape == "zeros":
        x[:, ::2] = -0.0
    elif shape == "steps":
        x[:] = np.floor(i / 64) % 37
    t = torch.from_numpy(x).to(DT[dtype]).cuda()
    tokens = torch.tensor([0, vocab - 1, 2], dtype=torch.int32, device="cuda")
    with np.errstate(all="ignore"):
        check(t, tokens, 1.0, min(vocab, 20))
        check(t, tokens, 1.0, min(vocab, 32))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", range(9))
def test_rows_at_every_alignment(off, dtype):
    """Rows that start anywhere within 16 bytes, with a row stride past their end; NaN around them is not read."""
    r = np.random.RandomState(off)
    rows, vocab = 6, 2051
    buf = torch.full((rows, vocab + 19), float("nan"), dtype=DT[dtype], device="cuda")
    buf[:, off:off + vocab] = logits(r, rows, vocab, dtype)
    tokens = torch.from_numpy(r.randint(0, vocab, rows).astype(np.int32)).cuda()
    check(buf[:, off:off + vocab], tokens, 1.0, 7)
    grad(buf[:, off:off + vocab], tokens, 1.0, r)


def grad(x, tokens, scale, r, parts="plh", dlogits=None):
    rows = x.size(0)
    X = f64(x)
    s = aq.aq_token_logprobs(x, tokens, scale=scale)
    g = {n: torch.from_numpy(r.standard_normal(rows).astype(np.float32)).cuda() for n in parts}
    d = aq.aq_token_logprobs_backward(x, tokens, s.lse, s.entropy if "h" in parts else None, g.get("p"), dentropy=g.get("h"), dlse=g.get("l"),
                                      scale=scale, dlogits=dlogits)
    assert d.dtype == x.dtype and d.shape == x.shape
    sc = np.float64(np.float32(scale))
    ref, size = serving.token_scores_backward(X, tokens.cpu().numpy(), f64(s.lse), f64(s.entropy), f64(g.get("p")), f64(g.get("h")), f64(g.get("l")), sc)
    with np.errstate(invalid="ignore"):
        logp = np.abs(np.nan_to_num(X * sc - f64(s.lse)[:, None], posinf=0, neginf=0))
    same(f64(d), ref, torch.finfo(x.dtype).eps / 2 * np.abs(ref) + 2.0 ** -20 * (1 + logp) * size + 1e-37)
    return d


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,scale,parts", [
    (1, 1, 1.0, "plh"), (3, 2, 1.0, "p"), (2, 7, 0.5, "h"), (5, 33, 2.0, "l"), (7, 1025, 1.25, "ph"), (200, 4097, 0.7, "plh"),
    (2, 32003, 1.0, "p"), (1, 262144, 1.0, "plh"), (40, 50257, 1.0, "p"), (900, 300, 1.0, "plh"),
])
def test_gradient(rows, vocab, scale, parts, dtype):
    r = np.random.RandomState(rows + vocab)
    x = logits(r, rows, vocab, dtype)
    tokens = torch.from_numpy(r.randint(0, vocab, rows).astype(np.int32)).cuda()
    if rows > 2:
        tokens[1], tokens[2] = -1, vocab
    want = grad(x, tokens, scale, np.random.RandomState(1), parts)
    # into a buffer whose rows start elsewhere, and in place
    buf = torch.full((rows, vocab + 3), 5.0, dtype=x.dtype, device="cuda")
    grad(x, tokens, scale, np.random.RandomState(1), parts, dlogits=buf[:, 2:vocab + 2])
    assert torch.equal(buf[:, 2:vocab + 2], want) and (buf[:, :2] == 5).all() and (buf[:, -1] == 5).all()
    mine = x.clone()
    s = aq.aq_token_logprobs(x, tokens, scale=scale)
    g = torch.ones(rows, device="cuda")
    apart = aq.aq_token_logprobs_backward(x, tokens, s.lse, None, g, scale=scale)
    assert aq.aq_token_logprobs_backward(mine, tokens, s.lse, None, g, scale=scale, dlogits=mine) is mine and torch.equal(mine, apart)


def test_gradient_of_special_rows():
    """Masked words have none; a row of nothing but -inf has zeros; NaN stays in its row."""
    x = torch.zeros(4, 50, device="cuda")
    x[0, 10:] = float("-inf")
    x[1] = float("-inf")
    x[2, 7] = float("nan")
    x[3, :] = torch.finfo(torch.float32).min
    x[3, 4] = 1.0
    tokens = torch.tensor([3, 3, 3, 4], dtype=torch.int32, device="cuda")
    s = aq.aq_token_logprobs(x, tokens)
    one = torch.ones(4, device="cuda")
    d = aq.aq_token_logprobs_backward(x, tokens, s.lse, s.entropy, one, dentropy=one, dlse=one)
    assert (d[0, 10:] == 0).all() and torch.isfinite(d[0]).all() and (d[1] == 0).all() and torch.isnan(d[2]).all()
    assert (d[3, :4] == 0).all() and (d[3, 5:] == 0).all() and abs(float(d[3, 4]) - 1.0) < 1e-6


def test_rows_past_32_bits():
    """Logits of more than 2^32 bytes: the last rows are read and written where they lie."""
    vocab, rows = 262144, 8300
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    tokens = torch.full((rows,), 5, dtype=torch.int32, device="cuda")
    x[-1, 5], x[-1, 262143] = 20.0, 21.0
    s = aq.aq_token_logprobs(x, tokens, top=2)
    assert s.top_token[-1].tolist() == [262143, 5] and s.top_token[-2].tolist() == [0, 1]
    _, lse, _, _, _ = serving.token_scores(f64(x[-2:]), None)
    same(f64(s.lse[-2:]), lse, 2.0 ** -24 * (8 * 30 + 16 + 4096) + 2.0 ** -23 * lse)
    g = torch.zeros(rows, device="cuda")
    g[-1] = 1.0
    d = aq.aq_token_logprobs_backward(x, tokens, s.lse, None, g, dlogits=x)
    assert (d[:-1] == 0).all() and float(d[-1, 5]) > 0 > float(d[-1, 262143])


def test_captured():
    r = np.random.RandomState(3)
    x = logits(r, 9, 5000, "bf16")
    tokens = torch.from_numpy(r.randint(0, 5000, 9).astype(np.int32)).cuda()
    g = torch.ones(9, device="cuda")

    def both():
        s = aq.aq_token_logprobs(x, tokens, top=4)
        return [*s, aq.aq_token_logprobs_backward(x, tokens, s.lse, s.entropy, g, dentropy=g)]

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for _ in range(3):
        x.copy_(logits(r, 9, 5000, "bf16"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, both()))
