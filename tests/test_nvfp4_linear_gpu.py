"""aq_nvfp4_linear on the GPU against the float64 product of the dequantised weights.

Tolerance, per element: the output's bf16 rounding, 2^-8 |y|; fp32 sums over K and over the parts of K, (K + 16) 2^-23 of
sum |w||x| (2^-23: the matrix instruction may truncate); x in f16 under a power of two: an element keeps a unit of 2^-24 where
the largest is 2^15 or more, so it is off by at most 2^-40 of the token's largest, times sum |w|. On small whole numbers every
product and sum is exact, and so is the result.
"""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from oracle import nvfp4
from rank_weight_reconstruction_gb300 import synth
from helpers import bits, dev_theta, host_f64

pytestmark = pytest.mark.gpu

LAYOUT = {"linear": aq.AQ_SF_LINEAR, "128x4": aq.AQ_SF_128X4}


def weight(r, out, inp, layout="linear", g=0.01, pad=0, whole=False):
    """A random weight: (Nvfp4Weight, its values in float64). pad: bytes more than a row between rows of codes."""
    codes = r.randint(0, 16, (out, inp)).astype(np.uint8)
    sf = r.choice([0x38, 0x40, 0x30], (out, inp // 16)).astype(np.uint8) if whole else r.randint(0, 0x7f, (out, inp // 16)).astype(np.uint8)
    rows = np.full((out, inp // 2 + pad), 0x77, np.uint8)
    rows[:, :inp // 2] = nvfp4.pack(codes)
    q = torch.from_numpy(rows).cuda()[:, :inp // 2]
    held = sf if layout == "linear" else nvfp4.scales_128x4(sf)
    w = aq.Nvfp4Weight(q, torch.from_numpy(np.ascontiguousarray(held)).cuda(), torch.full((1,), g, dtype=torch.float32, device="cuda"), LAYOUT[layout])
    return w, nvfp4.dequantize(codes, sf, np.float32(g))


def tokens(r, M, inp, pad=0):
    x = r.standard_normal((M, inp + pad)).astype(np.float32) * np.exp(r.standard_normal((M, 1)).astype(np.float32))
    return torch.from_numpy(x).to(torch.bfloat16).cuda()[:, :inp]


def check(y, x, w):
    X = x.double().cpu().numpy()
    ref, size = X @ w.T, np.abs(X) @ np.abs(w).T
    K = X.shape[1]
    lost = 2.0 ** -40 * np.abs(X).max(1, keepdims=True) * np.abs(w).sum(1)[None]
    got = y.double().cpu().numpy()
    bad = ~(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (K + 16) * 2.0 ** -23 * size + lost + 1e-37)
    assert not bad.any(), (np.abs(got - ref).max(), np.argwhere(bad)[:4])


@pytest.mark.parametrize("layout", ["linear", "128x4"])
@pytest.mark.parametrize("M,out,inp", [
    (1, 1, 16), (1, 16, 16), (2, 17, 48), (1, 15, 128), (3, 130, 144), (8, 33, 112), (9, 257, 1168), (16, 64, 2048), (17, 100, 272),
    (32, 1000, 1152), (33, 48, 640), (70, 129, 336), (1, 1536, 1152), (5, 1152, 6912), (16, 1152, 6912), (1, 20000, 256), (4, 30001, 64),
])
def test_matches_the_product(M, out, inp, layout):
    r = np.random.RandomState(M + out + inp)
    w, values = weight(r, out, inp, layout)
    x = tokens(r, M, inp)
    y = aq.aq_nvfp4_linear(w, x)
    assert y.shape == (M, out) and y.dtype == torch.bfloat16
    check(y, x, values)
    assert torch.equal(aq.aq_nvfp4_linear(w, x), y)      # the order of the sums is fixed


@pytest.mark.parametrize("M,out,inp", [(32, 200, 21504), (16, 3000, 5376), (8, 40, 32768), (3, 20, 65536), (32, 24, 65536), (24, 5000, 4096)])
def test_long_rows(M, out, inp):
    """x of a call does not fit one CTA's shared memory, or not for 32 tokens at once."""
    r = np.random.RandomState(out)
    w, values = weight(r, out, inp)
    x = tokens(r, M, inp)
    check(aq.aq_nvfp4_linear(w, x), x, values)


@pytest.mark.parametrize("layout", ["linear", "128x4"])
@pytest.mark.parametrize("M,out,inp", [(1, 96, 1152), (7, 70, 272), (16, 512, 2048), (40, 33, 112)])
def test_whole_numbers_are_exact(M, out, inp, layout):
    """Whole x, scales 0.5, 1 and 2, g = 2: every sum is a multiple of 1/2 below 2^24, so only the final rounding is left."""
    r = np.random.RandomState(inp)
    w, values = weight(r, out, inp, layout, g=2.0, whole=True)
    x = torch.from_numpy(r.randint(-4, 5, (M, inp)).astype(np.float32)).to(torch.bfloat16).cuda()
    want = torch.from_numpy(x.double().cpu().numpy() @ values.T).to(torch.float32).to(torch.bfloat16)
    assert torch.equal(aq.aq_nvfp4_linear(w, x).cpu(), want)


@pytest.mark.parametrize("M", [1, 11, 32])
def test_several_weights_strides_and_slices(M):
    """Three weights with rows of codes apart by 8 bytes more than they hold, x and the outputs as slices: what lies around
    the outputs is left alone, and each output is the single call's, bit for bit where the plan is the same or to rounding."""
    r = np.random.RandomState(M)
    inp, outs = 272, (50, 1, 77)
    ws = [weight(r, o, inp, pad=8) for o in outs]
    x = tokens(r, M, inp, pad=24)
    buf = torch.full((M + 2, sum(outs) + 9), 7.0, dtype=torch.bfloat16, device="cuda")
    at, ys = 3, []
    for o in outs:
        ys.append(buf[1:M + 1, at:at + o])
        at += o
    got = aq.aq_nvfp4_linear_multi([w for w, _ in ws], x, ys=ys)
    for y, (_, values), mine in zip(got, ws, ys):
        assert y is mine
        check(y, x, values)
    around = buf.clone()
    around[1:M + 1, 3:3 + sum(outs)] = 7.0
    assert (around == 7.0).all()
    assert aq.aq_nvfp4_linear(ws[0][0], x[:0]).shape == (0, 50)


def test_what_the_precompute_makes():
    """W_eff quantised by aq_precompute_nvfp4 in both layouts, straight into the product: the same values, the same bits."""
    th = synth.make_theta(("nvfp4 linear",), 384, 320, 8)
    d = dev_theta(th)
    r = np.random.RandomState(0)
    x = tokens(r, 6, 320)
    ys = []
    for layout in (aq.AQ_SF_LINEAR, aq.AQ_SF_128X4):
        q, sf, g = aq.aq_precompute_nvfp4(d, sf_layout=layout)
        ys.append(aq.aq_nvfp4_linear(aq.Nvfp4Weight(q, sf, g, layout), x))
        if layout == aq.AQ_SF_LINEAR:
            check(ys[0], x, nvfp4.dequantize(nvfp4.unpack(q.cpu().numpy()), sf.cpu().numpy(), np.float32(g.item())))
    assert torch.equal(*ys)
    # against the unquantised weight the quantisation itself shows, and no more: E2M1 is off by a sixth of a value at most (from 5
    # to 4 or 6 the step is 2: 1/5), a block's scale by 2^-4
    w = host_f64(aq.aq_precompute(d))
    ref = x.double().cpu().numpy() @ w.T
    assert np.linalg.norm(host_f64(ys[0]) - ref) <= 0.27 * np.linalg.norm(ref)


def test_special_values_stay_where_they_are():
    r = np.random.RandomState(5)
    w, values = weight(r, 40, 160)
    x = tokens(r, 5, 160)
    want = aq.aq_nvfp4_linear(w, x)
    y = x.clone()
    y[1, 7], y[3, 100] = float("nan"), float("inf")
    got = aq.aq_nvfp4_linear(w, y)
    assert torch.equal(got[[0, 2, 4]], want[[0, 2, 4]])
    assert torch.isnan(got[1]).all()
    ref = np.sign(values[:, 100])             # an infinity keeps its sign, and makes NaN of a weight of zero
    g3 = got[3].double().cpu().numpy()
    assert all(np.isnan(a) if s == 0 else a == s * np.inf for a, s in zip(g3, ref))
    # a NaN among the scales: its row alone; with the next row's scales NaN too, nothing shows past a row's end
    sf = w.sf.clone()
    sf[9, 2] = 0x7f
    got = aq.aq_nvfp4_linear(aq.Nvfp4Weight(w.q, sf, w.global_scale, w.layout), x)
    keep = [i for i in range(40) if i != 9]
    assert torch.isnan(got[:, 9]).all() and torch.equal(got[:, keep], want[:, keep])


@pytest.mark.parametrize("size", [1e-38, 1e-30, 1e30, 3e38])
def test_sizes_of_x(size):
    """Tokens of very different sizes, at the ends of bf16's range, each at its own power of two."""
    r = np.random.RandomState(6)
    w, values = weight(r, 24, 256, g=1e-4)
    x = tokens(r, 4, 256)
    x = x / x.abs().amax(1, keepdim=True)
    x[2] = x[2].float().mul(size).to(torch.bfloat16)
    x[3] = 0
    y = aq.aq_nvfp4_linear(w, x)
    if size < 1e-35:     # products with numbers at the bottom of the range leave fp32's normal numbers: up to 2^-126 each, times g
        d = np.abs(host_f64(y)[2] - x[2].double().cpu().numpy() @ values.T)
        assert (d <= 2.0 ** -8 * np.abs(x[2].double().cpu().numpy() @ values.T) + 1e-37).all()
        check(y[[0, 1, 3]], x[[0, 1, 3]], values)
    else:
        check(y, x, values)
    assert (y[3] == 0).all()


def test_captured_with_other_calls_between():
    """Two products in one graph, replayed on new inputs; a call on another stream at the same time."""
    r = np.random.RandomState(7)
    (w1, v1), (w2, v2) = weight(r, 96, 128), weight(r, 128, 96)
    x = tokens(r, 5, 128)
    mid, y = torch.empty(5, 96, dtype=torch.bfloat16, device="cuda"), torch.empty(5, 128, dtype=torch.bfloat16, device="cuda")

    def both():
        aq.aq_nvfp4_linear(w1, x, y=mid)
        aq.aq_nvfp4_linear(w2, mid, y=y)

    both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        both()
    for _ in range(3):
        x.copy_(tokens(r, 5, 128))
        graph.replay()
        other = aq.aq_nvfp4_linear(w1, x, stream=side)
        torch.cuda.synchronize()
        check(mid, x, v1)
        check(y, mid, v2)
        assert torch.equal(other, mid)
    assert bits(y).any()
