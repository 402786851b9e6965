"""Pins of the oracle's head norms, token scores and their gradients (float64 numpy): closed forms and central differences."""
import numpy as np
import pytest

from oracle import serving

H = 1e-5


def differences(f, x):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += H
        dn[i] -= H
        d[i] = (f(up) - f(dn)) / (2 * H)
    return d


def test_norm_by_hand():
    """(3, 4) has a mean square of 12.5; a weight held as its distance from one doubles at 1."""
    y = serving.head_norm_rope(np.array([[[3.0, 4.0]]]), [0.0, 1.0], None, None, 0.0, offset=1.0)
    assert np.allclose(y[0, 0], [3 / 12.5 ** 0.5, 8 / 12.5 ** 0.5])


def test_norm_then_rotation():
    r = np.random.RandomState(0)
    x, w = r.randn(4, 3, 32), r.randn(32)
    f, _ = serving.rope_angles(16)
    y = serving.head_norm_rope(x, w, [0, 1, 2, 900], f, 1e-6, offset=1.0, layout="interleaved")
    assert np.allclose(y[0], x[0] / np.sqrt((x[0] ** 2).mean(-1, keepdims=True) + 1e-6) * (1 + w))
    assert np.allclose(serving.rope(y, [0, 1, 2, 900], f, 1.0, "interleaved", inverse=True),
                       serving.head_norm_rope(x, w, None, None, 1e-6, offset=1.0))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_norm_gradient_against_differences(layout):
    r = np.random.RandomState(1)
    x, w, dy = r.randn(3, 2, 16), 0.3 * r.randn(16), r.randn(3, 2, 16)
    pos, (f, mag) = [0, 5, 70], serving.rope_angles(8)
    args = dict(eps=1e-3, offset=1.0, magnitude=1.1, layout=layout)
    dx, dw, size, wsize = serving.head_norm_rope_backward(dy, x, w, pos, f, **args)
    assert np.allclose(dx, differences(lambda v: (serving.head_norm_rope(v, w, pos, f, **args) * dy).sum(), x), atol=1e-8)
    assert np.allclose(dw, differences(lambda v: (serving.head_norm_rope(x, v, pos, f, **args) * dy).sum(), w), atol=1e-8)
    assert (size >= np.abs(dx) * (1 - 1e-12)).all() and (wsize >= np.abs(dw) * (1 - 1e-12)).all()


def test_scores_of_a_uniform_row():
    lp, lse, h, tl, tt = serving.token_scores(np.full((1, 8), 3.0), [5], scale=2.0, top=3)
    assert np.allclose([lp[0], lse[0], h[0]], [-np.log(8), 6 + np.log(8), np.log(8)])
    assert tt[0].tolist() == [0, 1, 2] and np.allclose(tl, -np.log(8))


def test_scores_of_special_rows():
    x = np.array([[-np.inf, 0.0, -np.inf], [-np.inf] * 3, [np.nan, 1.0, -np.inf], [np.inf, 1.0, 2.0]])
    lp, lse, h, tl, tt = serving.token_scores(x, [1, 0, 1, 7], top=3)
    assert lp[0] == 0 and lse[0] == 0 and h[0] == 0 and tt[0].tolist() == [1, 0, 2]
    assert lp[1] == -np.inf and lse[1] == -np.inf and h[1] == 0 and tt[1].tolist() == [0, 1, 2]
    assert np.isnan(lp[2]) and np.isnan(lse[2]) and tt[2].tolist() == [1, 2, 0]
    assert lp[3] == 0 and np.isnan(lse[3]) and np.isnan(tl[3]).all() and tt[3].tolist() == [0, 2, 1]


def test_scores_gradient_against_differences():
    r = np.random.RandomState(2)
    x, tok = 2 * r.randn(3, 11), np.array([4, -1, 0])
    gp, gh, gl = r.randn(3), r.randn(3), r.randn(3)

    def loss(v):
        lp, lse, h, _, _ = serving.token_scores(v, tok, scale=0.7)
        return (gp * lp + gh * h + gl * lse).sum()

    _, lse, h, _, _ = serving.token_scores(x, tok, scale=0.7)
    d, size = serving.token_scores_backward(x, tok, lse, h, gp, gh, gl, scale=0.7)
    assert np.allclose(d, differences(loss, x), atol=1e-8)
    assert (size >= np.abs(d) * (1 - 1e-9)).all()


def test_scores_of_a_row_at_the_types_lowest_value():
    """Equal words are equally likely whatever their value: the difference is taken before the sum's logarithm is added."""
    lp, lse, h, _, _ = serving.token_scores(np.full((1, 9), -3.4e38), [2])
    assert np.allclose([lp[0], h[0]], [-np.log(9), np.log(9)]) and lse[0] == -3.4e38
