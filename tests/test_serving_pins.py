"""Pins of the serving oracle (float64 numpy): properties that the definitions fix, so that the GPU tests
compare against something checked by itself."""
import numpy as np
import pytest

from oracle import serving


def _rng(*key):
    return np.random.RandomState(sum(ord(c) * 31 for c in str(key)))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_keeps_lengths_and_relative_positions(layout):
    """A rotation keeps the norm, its inverse undoes it, and the product of a rotated query and key depends on
    the difference of their positions alone; what lies past rotary_dim passes through."""
    r = _rng("rope", layout)
    f, mag = serving.rope_angles(32)
    x = r.randn(5, 3, 48)
    pos = np.array([0, 1, 7, 1000, 123456])
    y = serving.rope(x, pos, f, mag, layout)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-12)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
    assert np.allclose(serving.rope(y, pos, f, mag, layout, inverse=True), x, atol=1e-12)
    q, k = r.randn(1, 1, 32), r.randn(1, 1, 32)
    dots = [float((serving.rope(q, [a + d], f, 1.0, layout) * serving.rope(k, [a], f, 1.0, layout)).sum())
            for d in (3,) for a in (0, 10, 5000)]
    assert np.allclose(dots, dots[0], atol=1e-9)


def test_rotation_by_hand():
    """One pair at one radian a position: position 1 turns (1, 0) to (cos 1, sin 1)."""
    y = serving.rope(np.array([[[1.0, 0.0]]]), [1], np.array([1.0]))
    assert np.allclose(y[0, 0], [np.cos(1), np.sin(1)])


def test_long_context_rules():
    f, _ = serving.rope_angles(64)
    lin, m = serving.rope_angles(64, rule="linear", factor=4.0)
    assert np.allclose(lin * 4, f) and m == 1.0
    ntk, _ = serving.rope_angles(64, rule="ntk", factor=4.0)
    assert np.isclose(ntk[0], f[0]) and np.isclose(ntk[-1] * 4.0, f[-1])   # the slowest pair is interpolated fully
    for rule in ("yarn", "wavelength"):
        g, m = serving.rope_angles(64, rule=rule, factor=8.0, original_len=4096)
        assert np.isclose(g[0], f[0]) and np.isclose(g[-1] * 8.0, f[-1])
        assert np.all(g <= f * (1 + 1e-12)) and np.all(g >= f / 8 * (1 - 1e-12))
    assert np.isclose(serving.rope_angles(64, rule="yarn", factor=8.0, original_len=4096)[1], 0.1 * np.log(8) + 1)


def test_e4m3_rounding_against_torch():
    torch = pytest.importorskip("torch")
    assert serving.e4m3_values()[-1] == 448.0 and serving.e4m3_values()[1] == 2.0 ** -9
    x = np.concatenate([np.linspace(-448, 448, 40001), serving.e4m3_values(), -serving.e4m3_values(),
                        (serving.e4m3_values()[1:] + serving.e4m3_values()[:-1]) / 2, [2.0 ** -10, 1e-30]])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(serving.e4m3_round(x), want)
    assert serving.e4m3_round(1e9) == 448.0


def test_attention_row_pins():
    r = _rng("attn")
    k, v, q = r.randn(9, 4), r.randn(9, 4), r.randn(4)
    every = np.ones(9, bool)
    # equal scores: the mean of the values; one key: its value; nothing seen: zeros and -inf
    o, lse, _ = serving.attention_row(np.zeros(4), k, v, every, 1.0)
    assert np.allclose(o, v.mean(0)) and np.isclose(lse, np.log(9))
    one = np.arange(9) == 3
    assert np.allclose(serving.attention_row(q, k, v, one, 0.5)[0], v[3])
    o, lse, _ = serving.attention_row(q, k, v, ~every, 1.0)
    assert not o.any() and lse == -np.inf
    # masked keys take no part, whatever they hold
    bad_k, bad_v = k.copy(), v.copy()
    bad_k[3], bad_v[3] = np.nan, np.inf
    assert np.allclose(serving.attention_row(q, bad_k, bad_v, ~one, 1.0)[0], serving.attention_row(q, k, v, ~one, 1.0)[0])


def test_seen_keys_by_hand():
    s = serving.seen_keys(3, 3, 1)
    assert s.tolist() == [True, True, True, True, True, False]
    s = serving.seen_keys(3, 3, 2, mask_bits=[True, False, True], depth=[0, 0, 1])
    assert s.tolist() == [True, True, True, True, False, True]
    # window 2 at position 3 + 1: keys at positions 3 and 4 alone (drafted key 0 at 3, itself at 4)
    s = serving.seen_keys(3, 3, 2, mask_bits=[True, False, True], depth=[0, 0, 1], window=2)
    assert s.tolist() == [False, False, False, True, False, True]
    assert serving.seen_keys(5, 1, 0, window=1).tolist() == [False] * 5 + [True]


def _softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return e / e.sum(-1, keepdims=True)


@pytest.mark.parametrize("drafts", ["chain", "siblings", "certain"])
def test_verification_keeps_the_targets_distribution(drafts):
    """The first token that comes out (the first accepted draft, or the draw) is distributed as the target's
    row, however the drafts were made: frequencies within five standard deviations."""
    r = np.random.RandomState(5)
    V, n, N = 6, 2, 20000
    p, q = _softmax(r.randn(n + 1, V) * 1.5), _softmax(r.randn(n + 1, V) * 1.5)
    parent = [-1, 0] if drafts == "chain" else [-1, -1]
    counts = np.zeros(V)
    for _ in range(N):
        u, noise = r.rand(n), r.exponential(size=V)
        if drafts == "certain":
            tokens = [2, 4]
        elif drafts == "chain":
            tokens = [r.choice(V, p=q[0]), 0]
            tokens[1] = r.choice(V, p=q[1])
        else:
            tokens = [r.choice(V, p=q[0]), r.choice(V, p=q[0])]
        path, token, _ = serving.verify(tokens, parent, p, u, noise, q=None if drafts == "certain" else q)
        counts[tokens[path[0]] if path else token] += 1
    assert np.all(np.abs(counts / N - p[0]) < 5 * np.sqrt(p[0] * (1 - p[0]) / N))


def test_verification_limits():
    V = 4
    p = np.full((3, V), 0.25)
    # p equal to q: everything is accepted, and the draw is from the last row
    path, token, _ = serving.verify([1, 2], None, p, [0.99, 0.99], [1, 1, 0.5, 1], q=p)
    assert path == [0, 1] and token == 2
    # a token the target excludes is refused, and its residual excludes it
    p0 = np.array([[0.5, 0.0, 0.5, 0.0]] * 3)
    path, token, _ = serving.verify([1, 2], None, p0, [0.0, 0.5], [9, 1e-9, 1, 1])
    assert path == [] and token == 2
    # the walk ends at the cap, and its draw is from that row in full
    assert serving.verify([1, 2], None, p, [0.0, 0.0], [1, 1, 1, 0.5], cap=1)[:2] == ([0], 3)


@pytest.mark.parametrize("q_given", [True, False])
def test_padded_nodes_keep_the_targets_distribution(q_given):
    """Nodes without a token (-1) are not there: alone, the draw is the target's; beside a real draft, as without them."""
    r = np.random.RandomState(8)
    V, n = 5, 3
    p, q = _softmax(r.randn(n + 1, V) * 1.5), _softmax(r.randn(n + 1, V) * 1.5)
    for _ in range(200):
        u, noise = r.rand(n), r.exponential(size=V)
        Q = q if q_given else None
        path, token, _ = serving.verify([-1, V, -7], [-1, -1, 1], p, u, noise, q=Q)
        assert path == [] and token == int((p[0] / noise).argmax())
        x = int(r.choice(V, p=q[0]))
        padded = serving.verify([-1, x, V], [-1, -1, -1], p, u, noise, q=Q)
        plain = serving.verify([x], [-1], p[[0, 2]], u[1:2], noise, q=None if Q is None else q[[0, 2]])
        assert [1] * len(plain[0]) == padded[0] and padded[1] == plain[1]
