"""Head norms with the rotation, their gradient, and the cache's write with norms, on the GPU against the float64 oracle.

Tolerances: the output's bf16 rounding, 2^-8 |y|, and the fp32 evaluation: a sum of D squares in a tree of 16 and four levels
(20 x 2^-24 of the mean, half of it on its root), rsqrt and three products (6 x 2^-24), the rotation's 1e-6: below 4e-6 of the terms'
absolute values. The weights' gradients are fp32 sums of N terms, each off by 4e-6 of itself, in chains of at most N: (4e-6 + N 2^-24)
of the terms' absolute values."""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from oracle import serving

pytestmark = pytest.mark.gpu

EPS = 1e-6


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(r, *shape, by=1.0):
    return torch.from_numpy((by * r.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16).cuda()


def layout_of(name):
    return aq.AQ_ROPE_HALF if name == "half" else aq.AQ_ROPE_INTERLEAVED


def head_ok(got, x, w, pos, rot, layout, offset=1.0, eps=EPS):
    angles = None if rot is None else serving.rope_angles(rot)[0]
    ref = serving.head_norm_rope(f64(x), None if w is None else f64(w), pos, angles, eps, offset, layout=layout)
    flat = np.abs(serving.head_norm_rope(f64(x), None if w is None else f64(w), None, None, eps, offset))
    size = flat.copy()
    if rot is not None:
        n = rot // 2
        lo, hi = (slice(0, n), slice(n, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
        size[..., lo] = size[..., hi] = flat[..., lo] + flat[..., hi]
    d = np.abs(f64(got) - ref)
    bad = ~(d <= 2.0 ** -8 * np.abs(ref) + 4e-6 * size)
    assert not bad.any(), (float(d.max()), np.argwhere(bad)[:4])


SHAPES = [(1, 1, 1, 16, 16, "half"), (1, 4, 1, 256, 256, "half"), (5, 3, 2, 64, 16, "interleaved"), (33, 7, 7, 80, 48, "half"),
          (130, 2, 1, 128, 128, "interleaved"), (257, 5, 1, 96, 96, "half"), (64, 1, 1, 48, 16, "half"), (1000, 16, 4, 128, 64, "half"),
          (700, 33, 3, 32, 32, "interleaved"), (3001, 8, 8, 64, None, "half"), (2, 40, 8, 240, 240, "interleaved")]


@pytest.mark.parametrize("T,hq,hk,D,rot,layout", SHAPES)
def test_forward(T, hq, hk, D, rot, layout):
    r = np.random.RandomState(T + hq + D)
    q, k, wq, wk = randn(r, T, hq, D, by=3.0), randn(r, T, hk, D, by=0.01), randn(r, D, by=0.4), randn(r, D)
    pos = r.randint(0, 1 << 20, T).astype(np.int32)
    rope = None if rot is None else aq.rope_frequencies(rot, layout=layout_of(layout))
    p = torch.from_numpy(pos).cuda()
    qo, ko = aq.aq_qk_norm_rope(q, k, aq.HeadNorm(wq, EPS, 1.0), aq.HeadNorm(wk, 1e-3), rope, p if rope else None)
    head_ok(qo, q, wq, pos, rot, layout)
    head_ok(ko, k, wk, pos, rot, layout, offset=0.0, eps=1e-3)
    alone, none = aq.aq_qk_norm_rope(q, q_norm=aq.HeadNorm(None, EPS), rope=rope, pos=p)
    assert none is None
    head_ok(alone, q, None, pos, rot, layout)
    # without norms it is the rotation, bit for bit
    if rope:
        plain, also = aq.aq_qk_norm_rope(q, k, rope=rope, pos=p)
        assert torch.equal(plain, aq.aq_rope(rope, p, q)) and torch.equal(also, aq.aq_rope(rope, p, k))


def test_strides_and_in_place():
    """q and k as slices of one stacked output, in place and into heads-outermost outputs; nothing else is touched."""
    r = np.random.RandomState(4)
    T, hq, hk, D = 37, 6, 2, 64
    rope, pos = aq.rope_frequencies(D), torch.arange(T, dtype=torch.int32, device="cuda") * 100
    wq, wk = randn(r, D), randn(r, D)
    norms = aq.HeadNorm(wq, EPS, 1.0), aq.HeadNorm(wk, EPS, 1.0)
    qkv = randn(r, T, (hq + 2 * hk) * D + 8)
    before = qkv.clone()
    q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hk) * D].unflatten(1, (hk, D))
    want = aq.aq_qk_norm_rope(q.clone(), k.clone(), *norms, rope, pos)
    qo = torch.full((hq, T, D), float("nan"), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    aq.aq_qk_norm_rope(q, k, *norms, rope, pos, q_out=qo)
    assert torch.equal(qo, want[0]) and torch.equal(qkv, before)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, b = aq.aq_qk_norm_rope(q, k, *norms, rope, pos, q_out=q, k_out=k, stream=side)
    side.synchronize()
    assert a is q and b is k and torch.equal(q, want[0]) and torch.equal(k, want[1])
    qkv[:, :(hq + hk) * D] = before[:, :(hq + hk) * D]
    assert torch.equal(qkv, before)
    e, f = aq.aq_qk_norm_rope(q[:0], k[:0], *norms, rope, pos[:0])
    assert e.shape == (0, hq, D) and f.shape == (0, hk, D)


@pytest.mark.parametrize("by", [0.0, 1e-30, 1e15, 1e19, 2e38])
def test_sizes(by):
    """Heads whose squares leave fp32 at either end: a large head is normed like any other, a small one shrinks under eps."""
    r = np.random.RandomState(5)
    x = (randn(r, 3, 2, 64) / 4).clamp(-1, 1)
    x[1] = (x[1].double() * by).to(torch.bfloat16)
    y, _ = aq.aq_qk_norm_rope(x, q_norm=aq.HeadNorm(None, EPS))
    head_ok(y, x, None, None, None, "half")
    dy = randn(r, 3, 2, 64)
    dx, _, _, _ = aq.aq_qk_norm_rope_backward(dy, None, x, None, aq.HeadNorm(None, EPS), None)
    ref, _, size, _ = serving.head_norm_rope_backward(f64(dy), f64(x), None, None, None, EPS)
    # below the normal numbers a product is off by 2^-149 and a bf16 value by 2^-134
    assert (np.abs(f64(dx) - ref) <= 2.0 ** -8 * np.abs(ref) + 4e-6 * size + 2.0 ** -133).all()


def test_special_values():
    """A NaN or an infinity stays in its head."""
    r = np.random.RandomState(6)
    x, w = randn(r, 4, 3, 128), randn(r, 128)
    n = aq.HeadNorm(w, EPS)
    want, _ = aq.aq_qk_norm_rope(x, q_norm=n)
    y = x.clone()
    y[1, 2, 5], y[2, 0, 77] = float("nan"), float("-inf")
    got, _ = aq.aq_qk_norm_rope(y, q_norm=n)
    assert torch.isnan(got[1, 2]).all() and torch.isnan(got[2, 0, 77])
    rest = torch.ones(4, 3, dtype=torch.bool, device="cuda")
    rest[1, 2] = rest[2, 0] = False
    assert torch.equal(got[rest], want[rest])


@pytest.mark.parametrize("kind", [aq.AQ_KV_BF16, aq.AQ_KV_E4M3], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("T,hq,hk,D,rot", [(1, 4, 1, 256, 256), (5, 6, 2, 80, 32), (130, 32, 8, 128, 128), (67, 2, 1, 64, None)])
def test_cache_write(T, hq, hk, D, rot, kind):
    """The write with norms is the norms, then the write: queries bit for bit; keys to one rounding, which the norm's own bf16
    output has more than the cache's; values bit for bit. A slot outside the cache writes nothing."""
    r = np.random.RandomState(T + D)
    qkv = randn(r, T, (hq + 2 * hk) * D, by=2.0)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([hq * D, hk * D, hk * D], 1))
    norms = aq.HeadNorm(randn(r, D), EPS, 1.0), aq.HeadNorm(randn(r, D), EPS, 1.0)
    rope = None if rot is None else aq.rope_frequencies(rot)
    pos = torch.from_numpy(r.randint(0, 9999, T).astype(np.int32)).cuda()
    slots = torch.randperm(160, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))[:T].contiguous()
    cache, ref = aq.KvCache.empty(10, 16, hk, D, kind), aq.KvCache.empty(10, 16, hk, D, kind)
    for c in (cache, ref):
        for t in (c.k, c.v, c.k_scale, c.v_scale):
            if t is not None:
                t.zero_()
    qo = aq.aq_kv_write(cache, k, v, slots, rope=rope, pos=pos, q=q, q_norm=norms[0], k_norm=norms[1])
    qn, kn = aq.aq_qk_norm_rope(q, k, *norms, rope, pos)
    aq.aq_kv_write(ref, kn, v, slots)
    assert torch.equal(qo, qn)
    assert torch.equal(cache.v, ref.v)
    got, want = aq.aq_kv_read(cache, slots)[0], aq.aq_kv_read(ref, slots)[0]
    if kind == aq.AQ_KV_BF16:
        assert torch.equal(got, want)
    else:   # both half an E4M3 step from the number they quantise (2^-4, 2^-10 of the scale below the normal codes), whose bf16 form is 2^-8 off, read back in bf16
        top = f64(want).__abs__().max(-1, keepdims=True)
        assert (np.abs(f64(got) - f64(want)) <= (2.0 ** -3 + 2.0 ** -6) * np.abs(f64(want)) + top * 2.0 ** -17 * 1.1).all()
        exact = serving.head_norm_rope(f64(k), f64(norms[1].weight), pos.cpu().numpy(), None if rot is None else serving.rope_angles(rot)[0], EPS, 1.0)
        step = np.abs(exact).max(-1, keepdims=True) / 448
        assert (np.abs(f64(got) - exact) <= (2.0 ** -4 + 2.0 ** -8 + 1e-4) * np.abs(exact) + 2.0 ** -10 * step * 1.01).all()
    only = aq.KvCache.empty(10, 16, hk, D, kind)
    for t in (only.k, only.v, only.k_scale, only.v_scale):
        if t is not None:
            t.fill_(3)
    aq.aq_kv_write(only, k, v, torch.full_like(slots, -1), rope=rope, pos=pos, k_norm=norms[1])
    assert all((t == 3).all() for t in (only.k, only.v))


@pytest.mark.parametrize("T,hq,hk,D,rot,layout", SHAPES)
def test_backward(T, hq, hk, D, rot, layout):
    r = np.random.RandomState(T + hk + D)
    q, k, wq, wk = randn(r, T, hq, D, by=2.0), randn(r, T, hk, D, by=0.1), randn(r, D, by=0.4), randn(r, D)
    dqo, dko = randn(r, T, hq, D), randn(r, hk, T, D).transpose(0, 1)
    pos = r.randint(0, 1 << 20, T).astype(np.int32)
    rope = None if rot is None else aq.rope_frequencies(rot, layout=layout_of(layout))
    p = torch.from_numpy(pos).cuda() if rope else None
    norms = aq.HeadNorm(wq, EPS, 1.0), aq.HeadNorm(wk, 1e-3)
    got = aq.aq_qk_norm_rope_backward(dqo, dko, q, k, *norms, rope, p)
    angles = None if rot is None else serving.rope_angles(rot)[0]
    for i, (dy, x, w, eps, off) in enumerate([(dqo, q, wq, EPS, 1.0), (dko, k, wk, 1e-3, 0.0)]):
        dx, dw, size, wsize = serving.head_norm_rope_backward(f64(dy), f64(x), f64(w), pos, angles, eps, off, layout=layout)
        # a turned gradient's error is of its pair: twice the terms at most
        wide = size + np.abs(size).max(-1, keepdims=True)
        d = np.abs(f64(got[i]) - dx)
        assert (d <= 2.0 ** -8 * np.abs(dx) + 4e-6 * wide).all(), d.max()
        n = T * x.size(1)
        assert got[2 + i].dtype == torch.float32
        err = np.abs(f64(got[2 + i]) - dw)
        assert (err <= (8e-6 + n * 2.0 ** -24) * (wsize + wsize.max())).all(), err.max()
    again = aq.aq_qk_norm_rope_backward(dqo, dko, q, k, *norms, rope, p)
    assert all(torch.equal(a, b) for a, b in zip(got, again))      # the sums' order is fixed
    # in place of the output's gradient, q alone, and without a weight
    mine = dqo.clone()
    dq, dk, dqw, dkw = aq.aq_qk_norm_rope_backward(mine, None, q, None, norms[0], None, rope, p, dq=mine)
    assert dq is mine and dk is None and dkw is None and torch.equal(dq, got[0])
    none = aq.aq_qk_norm_rope_backward(dqo, None, q, None, aq.HeadNorm(None, EPS), None, rope, p)
    assert none[1:] == (None, None, None)
    head_dx, _, size, _ = serving.head_norm_rope_backward(f64(dqo), f64(q), None, pos, angles, EPS, layout=layout)
    assert (np.abs(f64(none[0]) - head_dx) <= 2.0 ** -8 * np.abs(head_dx) + 4e-6 * (size + size.max(-1, keepdims=True))).all()


def test_backward_of_nothing():
    """No tokens: the weights' gradients are zeros."""
    x = torch.empty(0, 3, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    dq, dk, dqw, dkw = aq.aq_qk_norm_rope_backward(x, x, x, x, aq.HeadNorm(w), aq.HeadNorm(w))
    assert dq.shape == x.shape and (dqw == 0).all() and (dkw == 0).all()


def test_two_graphs_with_a_workspace_each():
    """Captured backward passes with workspaces of their own, replayed at once on two streams."""
    r = np.random.RandomState(9)
    T, h, D = 300, 4, 128
    w = randn(r, D)
    n = aq.HeadNorm(w, EPS, 1.0)
    sets = [(randn(r, T, h, D), randn(r, T, h, D)) for _ in range(2)]
    want = [aq.aq_qk_norm_rope_backward(dy, None, x, None, n, None) for dy, x in sets]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for (dy, x), st in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            outs.append(aq.aq_qk_norm_rope_backward(dy, None, x, None, n, None))
        graphs.append(g)
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
