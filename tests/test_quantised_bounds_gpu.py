"""Where the bounds that the header states begin and end: a norm's eps beside heads whose squares leave fp32, x whose elements differ by
2^32 and more, and the C entry for a single weight."""
import ctypes

import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from oracle import nvfp4, serving
from rank_weight_reconstruction_gb300 import binding as b
import test_head_norm_gpu as norms
import test_nvfp4_linear_gpu as products

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** 50, 2.0 ** 55, 2.0 ** 56, 2.0 ** 58])
@pytest.mark.parametrize("eps", [1e-6, 1e20, 9e29])
@pytest.mark.parametrize("D,hq", [(256, 3), (64, 8)])
def test_eps_of_large_heads(D, hq, eps, size):
    """eps counts whatever a head's size. The weight's gradient is fp32 and shows it: (8e-6 + N 2^-24) of the terms, as in the norms' own
    test. The input's is off by 4e-6 of its terms besides its rounding."""
    r = np.random.RandomState(D)
    T = 7
    x, dy, w = norms.randn(r, T, hq, D, by=1.5), norms.randn(r, T, hq, D), norms.randn(r, D)
    x = (x.double() * size).to(torch.bfloat16)
    n = aq.HeadNorm(w, eps, 1.0)
    norms.head_ok(aq.aq_qk_norm_rope(x, q_norm=n)[0], x, w, None, None, "half", eps=float(np.float32(eps)))
    dx, _, dw, _ = aq.aq_qk_norm_rope_backward(dy, None, x, None, n, None)
    ref, wref, terms, wterms = serving.head_norm_rope_backward(norms.f64(dy), norms.f64(x), norms.f64(w), None, None, float(np.float32(eps)), 1.0)
    assert (np.abs(norms.f64(dw) - wref) <= (8e-6 + T * hq * 2.0 ** -24) * wterms).all(), (np.abs(norms.f64(dw) - wref) / wterms).max()
    assert (np.abs(norms.f64(dx) - ref) <= 2.0 ** -8 * np.abs(ref) + 4e-6 * terms).all()


def muted(r, out, inp, M, cols):
    """A weight with codes of zero in `cols`, its values, and x between 1 and 2 with zeros there."""
    codes = r.randint(0, 16, (out, inp)).astype(np.uint8)
    codes[:, cols] = r.choice([0, 8], (out, len(cols))).astype(np.uint8)
    sf = r.randint(0x20, 0x60, (out, inp // 16)).astype(np.uint8)
    w = aq.Nvfp4Weight(torch.from_numpy(nvfp4.pack(codes)).cuda(), torch.from_numpy(sf).cuda(), torch.full((1,), 0.5, device="cuda"))
    x = torch.from_numpy(((1 + r.random_sample((M, inp))) * r.choice([-1, 1], (M, inp))).astype(np.float32)).clamp(-1.984375, 1.984375).to(torch.bfloat16).cuda()
    x[:, cols] = 0
    return w, nvfp4.dequantize(codes, sf, np.float32(0.5)), x


def apart(got, x, values, far, at):
    """Tolerance of the products' own test, and in the 256 of K around `at`, for tokens with 2^far there: elements between 1 and 2 are at
    2^(15 - far) and off by half of f16's lowest unit, 2^(far - 40) of their own scale, but by no more than themselves; those below f16's
    normal numbers, 2^-14, may enter a sum aligned as if they were that large: 2^(far - 29) times the unit of a sum."""
    X, W = products.host_f64(x), np.abs(values)
    K = X.shape[1]
    ref, size, hit = X @ values.T, np.abs(X) @ W.T, np.abs(X[:, at]) == 2.0 ** far
    near = slice(at // 256 * 256, at // 256 * 256 + 256)
    here = 2 * W[:, near].sum(1)[None] * hit[:, None]
    off = min(2.0 ** (far - 41), 1.0) * here if far > 32 else 0
    tol = 2.0 ** -8 * (np.abs(ref) + off) + (K + 16) * 2.0 ** -23 * size + off + 272 * min(2.0 ** (far - 52), 1.0) * here
    d = np.abs(products.host_f64(got) - ref)
    assert (d <= tol).all(), (d / tol).max()


@pytest.mark.parametrize("far", [20, 32, 34, 40, 60])
@pytest.mark.parametrize("M,out,inp,at", [(1, 200, 1152, 5), (8, 5000, 1024, 700), (5, 40, 6912, 6900), (32, 1000, 272, 260)])
def test_one_element_far_above_the_rest(M, out, inp, at, far):
    """In every other token, over codes of zero, so that the rest is all there is. Down to 2^-32 of it an element keeps its bits; further down
    it loses them, in this token and 256 of K alone."""
    r = np.random.RandomState(out + far)
    w, values, x = muted(r, out, inp, M, np.array([at]))
    x[::2, at] = 2.0 ** far
    apart(aq.aq_nvfp4_linear(w, x), x, values, far, at)


def test_the_single_weight_entry():
    """aq_nvfp4_linear of the C ABI is the call for several weights with one of them."""
    lib = b.load()
    r = np.random.RandomState(3)
    for layout in ("linear", "128x4"):
        w, values = products.weight(r, 130, 272, layout)
        x = products.tokens(r, 9, 272, pad=8)
        y = torch.full((9, 133), 7.0, dtype=torch.bfloat16, device="cuda")
        c = b.c_nvfp4_weight(w.q.data_ptr(), w.q.stride(0), w.sf.data_ptr(), w.global_scale.data_ptr(), w.layout, 130, 272)
        assert lib.aq_nvfp4_linear(ctypes.byref(c), x.data_ptr(), 9, x.stride(0), y.data_ptr(), y.stride(0), torch.cuda.current_stream().cuda_stream) == b.AQ_OK
        products.check(y[:, :130], x, values)
        assert torch.equal(y[:, :130], aq.aq_nvfp4_linear(w, x)) and (y[:, 130:] == 7).all()
