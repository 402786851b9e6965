"""NVFP4 products, head norms and token scores where their work is cut up: tiles that step from one block of scales to the next, rows of
K that end in half a chunk, CTAs without a part of K, many rows of few words, heads fewer than a warp's groups, offsets past 32 bits,
and two streams at once. Tolerances are those of the operators' own tests."""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from oracle import serving
import test_head_norm_gpu as norms
import test_nvfp4_linear_gpu as products
import test_scores_gpu as scores

pytestmark = pytest.mark.gpu


# ---- products ----
@pytest.mark.parametrize("layout", ["linear", "128x4"])
@pytest.mark.parametrize("M", [1, 8, 13, 32])
@pytest.mark.parametrize("out,inp", [(5000, 272), (2056, 384), (4100, 1152), (2600, 1936), (9000, 144), (9000, 128), (700, 5360), (3000, 6912)])
def test_many_tiles_and_ragged_ends(out, inp, M, layout):
    """K that ends 16 to 240 into its last chunk of 256, blocks of 128 rows in a tile's path, a last tile of 4 to 12 rows, and for the last
    two K slices of which the last holds nothing."""
    r = np.random.RandomState(out + M)
    w, values = products.weight(r, out, inp, layout)
    x = products.tokens(r, M, inp)
    products.check(aq.aq_nvfp4_linear(w, x), x, values)


@pytest.mark.parametrize("M", [1, 9])
@pytest.mark.parametrize("pad", [8, 16])
def test_rows_of_codes_on_8_bytes(M, pad):
    """Rows of codes that start on 8 bytes, and on 16 apart by more than they hold, for several weights whose tiles follow one another."""
    r = np.random.RandomState(M + pad)
    ws = [products.weight(r, o, 656, pad=pad) for o in (1600, 16, 2005)]
    x = products.tokens(r, M, 656)
    for y, (_, values) in zip(aq.aq_nvfp4_linear_multi([w for w, _ in ws], x), ws):
        products.check(y, x, values)


def test_nothing_behind_a_row_counts():
    """NaN scales behind the last of a row's (the layout's filling, or the row after a slice of rows), and NaN behind x's columns."""
    r = np.random.RandomState(8)
    for inp in (144, 208, 272, 1072):
        w, values = products.weight(r, 40, inp, "128x4")
        sf = w.sf.clone().view(-1)
        held = torch.zeros_like(sf)
        rows, cols = np.arange(40)[:, None], np.arange(inp // 16)[None]
        at = (rows // 128 * ((inp // 16 + 3) // 4) + cols // 4) * 512 + rows % 32 * 16 + rows % 128 // 32 * 4 + cols % 4
        held[torch.from_numpy(at.ravel()).cuda()] = 1
        sf[held == 0] = 0x7f
        x = products.tokens(r, 5, inp, pad=24)
        x.as_strided((5, 24), (inp + 24, 1), inp).fill_(float("nan"))
        products.check(aq.aq_nvfp4_linear(aq.Nvfp4Weight(w.q, sf, w.global_scale, aq.AQ_SF_128X4), x), x, values)
        w, values = products.weight(r, 40, inp)
        sf = torch.full((41, inp // 16), 0x7f, dtype=torch.uint8, device="cuda")
        sf[:40] = w.sf
        products.check(aq.aq_nvfp4_linear(aq.Nvfp4Weight(w.q, sf[:40], w.global_scale), x), x, values)


def test_products_past_32_bits():
    """Codes, and outputs, whose rows lie 2^27 bytes apart: past 2^32 from the 32nd row on."""
    r = np.random.RandomState(9)
    w, values = products.weight(r, 40, 528)
    far = torch.empty(40 << 27, dtype=torch.uint8, device="cuda")
    q = far.as_strided((40, 264), (1 << 27, 1), 64)
    q.copy_(w.q)
    x = products.tokens(r, 40, 528)
    products.check(aq.aq_nvfp4_linear(aq.Nvfp4Weight(q, w.sf, w.global_scale), x), x, values)
    y = far.view(torch.bfloat16).as_strided((40, 40), (1 << 26, 1), 4096)
    aq.aq_nvfp4_linear(w, x, y=y)
    products.check(y, x, values)


# ---- head norms ----
@pytest.mark.parametrize("T,hq,hk,D", [(9001, 1, 1, 16), (6003, 3, 1, 48), (5001, 2, 2, 80), (2500, 5, 2, 256), (20011, 1, 1, 128), (12001, 1, 1, 64),
                                       (9999, 2, 1, 64), (8001, 4, 1, 32), (7003, 1, 1, 256), (15001, 3, 1, 80)])
def test_more_tokens_than_the_grid_holds_in_place(T, hq, hk, D):
    r = np.random.RandomState(T)
    q, k, dq, dk = norms.randn(r, T, hq, D), norms.randn(r, T, hk, D), norms.randn(r, T, hq, D), norms.randn(r, T, hk, D)
    n = aq.HeadNorm(norms.randn(r, D), 1e-6, 1.0)
    rope, pos = aq.rope_frequencies(D), torch.from_numpy(r.randint(0, 1 << 20, T).astype(np.int32)).cuda()
    want, grads = aq.aq_qk_norm_rope(q, k, n, n, rope, pos), aq.aq_qk_norm_rope_backward(dq, dk, q, k, n, n, rope, pos)
    norms.head_ok(want[0], q, n.weight, pos.cpu().numpy(), D, "half")
    norms.head_ok(want[1], k, n.weight, pos.cpu().numpy(), D, "half")
    mine = aq.aq_qk_norm_rope_backward(dq, dk, q, k, n, n, rope, pos, dq=dq, dk=dk)
    assert mine[0] is dq and mine[1] is dk and all(torch.equal(a, b) for a, b in zip(mine, grads))
    got = aq.aq_qk_norm_rope(q, k, n, n, rope, pos, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("T,hq,hk,D,rot,layout", [
    (12001, 1, 1, 64, 64, "half"), (9999, 4, 1, 128, 64, "interleaved"), (8001, 3, 2, 32, 16, "half"), (7003, 1, 1, 256, 256, "interleaved"),
    (15001, 2, 1, 80, 80, "half"), (5001, 1, 1, 16, None, "half"), (2003, 5, 3, 48, 48, "interleaved"),
    (8, 32, 8, 128, 128, "half"), (64, 4, 1, 128, 64, "half"), (65, 4, 1, 128, 128, "interleaved"), (16, 40, 8, 256, 256, "half"), (40, 3, 1, 80, 80, "interleaved"),
    (127, 1, 1, 64, 64, "half"), (512, 1, 1, 16, 16, "half"), (2, 1, 64, 32, 32, "half"),
])
def test_gradient_of_few_heads_or_few_tokens(T, hq, hk, D, rot, layout):
    norms.test_backward(T, hq, hk, D, rot, layout)


def test_heads_past_32_bits():
    """Tokens 2^31 elements apart, read and written there."""
    r = np.random.RandomState(2)
    far = torch.empty(3 << 31, dtype=torch.bfloat16, device="cuda")
    q = far.as_strided((3, 4, 64), (1 << 31, 64, 1), 256)
    q.copy_(norms.randn(r, 3, 4, 64))
    near, dy = q.clone(), norms.randn(r, 3, 4, 64)
    n, rope, pos = aq.HeadNorm(norms.randn(r, 64)), aq.rope_frequencies(64), torch.arange(3, dtype=torch.int32, device="cuda")
    want = aq.aq_qk_norm_rope(near, q_norm=n, rope=rope, pos=pos)[0]
    grads = aq.aq_qk_norm_rope_backward(dy, None, near, None, n, None, rope, pos)
    dx = far.as_strided((3, 4, 64), (1 << 31, 64, 1), 4096)
    got = aq.aq_qk_norm_rope_backward(dy, None, q, None, n, None, rope, pos, dq=dx)
    assert torch.equal(dx, grads[0]) and torch.equal(got[2], grads[2])
    aq.aq_qk_norm_rope(q, q_norm=n, rope=rope, pos=pos, q_out=q)
    assert torch.equal(q, want)


# ---- scores ----
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,vocab,top", [(600, 1, 1), (600, 257, 0), (1000, 3000, 5), (900, 8191, 16), (900, 8193, 17), (2500, 1000, 32), (2500, 16384, 20),
                                            (600, 16385, 3), (457, 65, 2), (950, 16385, 8), (1300, 32768, 16), (1300, 32769, 9), (1220, 20000, 8),
                                               (470, 9001, 32), (480, 50257, 5), (470, 65000, 21), (290, 20000, 0), (150, 33000, 0)])
def test_many_rows_of_few_words(rows, vocab, top, dtype):
    r = np.random.RandomState(rows + vocab)
    x = scores.logits(r, rows, vocab, dtype)
    tokens = torch.from_numpy(r.randint(0, vocab, rows).astype(np.int32)).cuda()
    a = scores.check(x, tokens, 0.8, top)
    assert all(u is v is None or torch.equal(u, v) for u, v in zip(a, aq.aq_token_logprobs(x, tokens, scale=0.8, top=top)))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [33, 2500, 9001, 18003])
def test_many_rows_that_are_hard(vocab, dtype):
    """As single rows of this kind: ties, rising words, few words above minus infinity, NaN and infinities, many rows of them."""
    r = np.random.RandomState(vocab)
    x = r.standard_normal((800, vocab)).astype(np.float32)
    i = np.arange(vocab, dtype=np.float32)
    x[0::8], x[1::8], x[2::8], x[3::8] = 2.5, i / vocab * 20, -np.inf, np.floor(i / 64) % 37
    for row in range(2, 800, 8):
        x[row, r.randint(0, vocab, row % 7)] = 1.0
    x[4::8, vocab // 3], x[5::8, vocab // 2], x[6::8] = np.nan, np.inf, torch.finfo(scores.DT[dtype]).min
    x[6::16, vocab // 4] = 0.0
    tokens = torch.from_numpy(r.randint(0, vocab, 800).astype(np.int32)).cuda()
    with np.errstate(all="ignore"):
        scores.check(torch.from_numpy(x).to(scores.DT[dtype]).cuda(), tokens, 1.0, 12)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("vocab", [40000, 262144])
def test_few_allowed_words(vocab, dtype):
    """A mask that leaves fewer words than are asked for, as many, a few more, and more than one CTA ranks at a time, all equal or not."""
    r = np.random.RandomState(vocab)
    x = np.full((10, vocab), -np.inf, np.float32)
    for row, left in enumerate((1, 19, 20, 21, 100, 511, 513, 1500)):
        x[row, r.choice(vocab, left, replace=False)] = r.standard_normal(left) if row % 2 else 3.0
    x[8, :700], x[9, -700:] = 1.0, np.linspace(0, 1, 700)
    tokens = torch.from_numpy(np.argmax(x, 1).astype(np.int32)).cuda()
    with np.errstate(all="ignore"):
        scores.check(torch.from_numpy(x).to(scores.DT[dtype]).cuda(), tokens, 1.0, 20)


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e4, 1e30])
def test_scales(scale):
    r = np.random.RandomState(6)
    for rows, vocab in ((3, 5000), (700, 300)):
        x = scores.logits(r, rows, vocab, "bf16")
        tokens = torch.from_numpy(r.randint(0, vocab, rows).astype(np.int32)).cuda()
        with np.errstate(all="ignore"):
            scores.check(x, tokens, scale, 6)


# ---- together ----
def test_two_streams_at_once():
    """Every call on two streams side by side, over and over, gives what it gives alone."""
    import test_norm_scores_streams_gpu as streams

    calls = streams.inputs()
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(10):
        for i, s in enumerate(side):
            for k in (list(calls) if (turn + i) % 2 else list(calls)[::-1]):
                got.append((k, calls[k](stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for k, out in got for a, b in zip(out, want[k]))


def test_one_graph_on_two_streams_of_it():
    """Calls that a graph runs side by side."""
    import test_norm_scores_streams_gpu as streams

    calls = streams.inputs()
    want = {k: f() for k, f in calls.items()}
    torch.cuda.synchronize()
    graph, side, got = torch.cuda.CUDAGraph(), torch.cuda.Stream(), []
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        for k in calls:
            got.append((k, calls[k]()))
        with torch.cuda.stream(side):
            for k in list(calls)[::-1]:
                got.append((k, calls[k]()))
        main.wait_stream(side)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for k, out in got for a, b in zip(out, want[k]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_scores_far_from_zero(dtype):
    """Rows whose values pass from where a weight's exponent is one fused product to where it is a difference (2^26 of log2 units), in
    either order within a row, and differences there that matter: only these, not the values' size, count."""
    r = np.random.RandomState(12)
    step = 2.0 ** 3 if dtype == "f32" else 2.0 ** 19
    x = np.empty((8, 6000), np.float64)
    for row in range(8):
        x[row] = (46500000 // step + r.randint(-40, 40, 6000)) * step * (-1) ** row
    x[4:] = np.sort(x[4:], 1)
    x[6:] = x[6:, ::-1]
    t = torch.from_numpy(x.astype(np.float32)).to(scores.DT[dtype]).cuda()
    tokens = torch.from_numpy(np.argmax(scores.f64(t), 1).astype(np.int32)).cuda()
    # of values near 2^26 the log probabilities and the entropy are as exact as of any others: a difference is exact, its product is not
    for scale in (1.0, 0.03125):
        s = aq.aq_token_logprobs(t, tokens, scale=scale, top=20)
        lp, lse, h, tl, tt = serving.token_scores(scores.f64(t), tokens.cpu().numpy(), np.float64(np.float32(scale)), 20)
        tol = 2.0 ** -24 * (8 * 30 + 16 + 4096)
        size = np.abs(tl)
        scores.same(scores.f64(s.logprob), lp, tol)
        scores.same(scores.f64(s.top_logprob), tl, tol + 2.0 ** -22 * size)
        scores.same(scores.f64(s.entropy), h, tol * (1 + h))
        scores.same(scores.f64(s.lse), lse, tol + 2.0 ** -23 * np.abs(lse))
        assert np.array_equal(s.top_token.cpu().numpy(), tt)
        d = aq.aq_token_logprobs_backward(t, tokens, s.lse, None, torch.ones(8, device="cuda"), scale=scale)
        assert torch.isfinite(d).all() and d.abs().max() <= 1


FIRST = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import rank_weight_reconstruction_gb300 as aq
r = torch.Generator(device="cuda").manual_seed(1)
byte = lambda *s: torch.randint(0, 0x70, s, generator=r, device="cuda", dtype=torch.uint8)
randn = lambda *s: torch.randn(*s, generator=r, device="cuda").to(torch.bfloat16)
w = aq.Nvfp4Weight(byte(200, 2048), byte(200, 256), torch.ones(1, device="cuda"))
x, h, dh, z, n = randn(9, 4096), randn(30, 2, 64), randn(30, 2, 64), randn(5, 70000), aq.HeadNorm(randn(64))
tok, one = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.ones(5, device="cuda")

def run():
    s = aq.aq_token_logprobs(z, tok, top=3)
    return [aq.aq_nvfp4_linear(w, x), aq.aq_qk_norm_rope(h, q_norm=n)[0], *aq.aq_qk_norm_rope_backward(dh, None, h, None, n, None)[::2], *s,
            aq.aq_token_logprobs_backward(z, tok, s.lse, None, one)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = run()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, run()))
print("captured")
"""


def test_first_calls_of_a_process_captured():
    """No call of these needs to have run before it is captured."""
    import pathlib
    import subprocess
    import sys

    root = str(pathlib.Path(__file__).resolve().parents[1])
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
