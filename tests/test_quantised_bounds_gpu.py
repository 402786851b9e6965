"""Where the bounds that the header states begin and end: a norm's eps beside heads whose squares leave fp32."""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from oracle import serving
import test_head_norm_gpu as norms

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
