"""The serving operators in float64 numpy, from their definitions: rotary positions, the quantised
key/value vector, attention of drafted tokens, and the verification of drafts."""
import numpy as np

E4M3_MAX = 448.0


def rope_angles(rotary_dim, base=10000.0, rule="none", factor=1.0, original_len=0.0, fast=32.0, slow=1.0):
    """Radians a position of each of rotary_dim / 2 pairs, and the magnitude."""
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    if rule == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2.0))
    f = base ** (-2.0 * i / rotary_dim)
    if rule == "linear":
        return f / factor, 1.0
    if rule == "yarn":
        def pair(turns):
            return rotary_dim * np.log(original_len / (2 * np.pi * turns)) / (2 * np.log(base))
        lo, hi = max(np.floor(pair(fast)), 0.0), min(np.ceil(pair(slow)), rotary_dim - 1.0)
        mix = np.clip((i - lo) / max(hi - lo, 1e-3), 0, 1)
        return (1 - mix) * f + mix * f / factor, 0.1 * np.log(factor) + 1.0
    if rule == "wavelength":
        keep = np.clip((original_len * f / (2 * np.pi) - slow) / (fast - slow), 0, 1)
        return keep * f + (1 - keep) * f / factor, 1.0
    return f, 1.0


def rope(x, pos, angles, magnitude=1.0, layout="half", inverse=False):
    """x [T, H, D]; the pairs' angles times pos, forward or back."""
    y = np.array(x, dtype=np.float64)
    n = len(angles)
    # positions times angles, reduced modulo a turn before they lose bits
    turn = np.mod(np.asarray(pos, np.float64)[:, None] * (np.asarray(angles, np.float64) / (2 * np.pi))[None], 1.0)
    c, s = np.cos(2 * np.pi * turn)[:, None] * magnitude, np.sin(2 * np.pi * turn)[:, None] * magnitude
    if inverse:
        s = -s
    lo = slice(0, n) if layout == "half" else slice(0, 2 * n, 2)
    hi = slice(n, 2 * n) if layout == "half" else slice(1, 2 * n, 2)
    a, b = y[..., lo].copy(), y[..., hi].copy()
    y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
    return y


def e4m3_values():
    """The 127 non-negative finite values of E4M3, in order of their codes."""
    codes = np.arange(127)
    e, m = codes >> 3, codes & 7
    return np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))


def e4m3_round(x):
    """Nearest E4M3 value, ties to the even code, saturating."""
    v = e4m3_values()
    a = np.minimum(np.abs(np.asarray(x, np.float64)), E4M3_MAX)
    hi = np.clip(np.searchsorted(v, a), 1, 126)
    lo = hi - 1
    d = (a - v[lo]) - (v[hi] - a)
    pick = np.where(d < 0, lo, np.where(d > 0, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.sign(x) * v[pick]


def seen_keys(ctx, T, i, mask_bits=None, depth=None, window=0):
    """Which of the ctx + T keys drafted token i of a sequence sees. mask_bits: [T] truth values of its row."""
    seen = np.zeros(ctx + T, dtype=bool)
    seen[:ctx] = True
    seen[ctx:] = np.arange(T) <= i if mask_bits is None else np.asarray(mask_bits, bool)
    d = np.arange(T) if depth is None or mask_bits is None else np.asarray(depth)
    if window > 0:
        at = np.concatenate([np.arange(ctx), ctx + d])
        seen &= (ctx + d[i]) - at < window
    return seen


def attention_row(q, k, v, seen, scale):
    """One row over keys k, v [n, D]: (output, lse, sum of p |v|). Nothing seen: zeros and -inf."""
    if not seen.any():
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1])
    s = (k[seen] @ q) * scale
    m = s.max()
    if m == -np.inf:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1])
    w = np.exp(s - m)
    total = w.sum()
    return (w @ v[seen]) / total, m + np.log(total), (w @ np.abs(v[seen])) / total


def verify(tokens, parent, p, u, noise, q=None, cap=None):
    """One sequence: tokens, parent [n], p (and q) [n + 1, V], u [n], noise [V]. Returns (path, next token,
    margin): margin is the smallest relative distance of any comparison from its tie."""
    n = len(tokens)
    cap = n if cap is None else cap
    parent = list(range(-1, n - 1)) if parent is None else list(parent)
    here, path, margin = -1, [], np.inf

    def near(a, b):
        nonlocal margin
        if max(abs(a), abs(b)) > 0:
            margin = min(margin, abs(a - b) / max(abs(a), abs(b)))

    while True:
        target = np.asarray(p[here + 1], np.float64)
        left, gone, moved = target.copy(), 0.0, False
        for c in range(here + 1, n) if len(path) < cap else ():
            if parent[c] != here:
                continue
            x = tokens[c]
            if not 0 <= x < len(target):      # no token: no draft
                continue
            bar = u[c] * (1.0 - gone if q is None else q[here + 1][x])
            near(bar, left[x])
            if bar < left[x]:
                path.append(c)
                here, moved = c, True
                break
            if q is not None:
                left = np.maximum(left - np.asarray(q[here + 1], np.float64), 0.0)
                left = left / left.sum() if left.sum() > 0 else left
            else:
                gone += left[x]
                left[x] = 0.0
        if not moved:
            break
    if not left.sum() > 0:
        left = target
    score = left / np.asarray(noise, np.float64)
    best = np.argsort(-score, kind="stable")[:2]
    if len(best) > 1:
        near(score[best[0]], score[best[1]])
    return path, int(best[0]), margin


def head_norm_rope(x, weight, pos, angles, eps, offset=0.0, magnitude=1.0, layout="half"):
    """x [T, H, D] normed head by head, times offset + weight (weight None: one), then rotated (angles None: not)."""
    x = np.asarray(x, np.float64)
    f = 1.0 if weight is None else offset + np.asarray(weight, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * f
    return y if angles is None else rope(y, pos, angles, magnitude, layout)


def head_norm_rope_backward(dy, x, weight, pos, angles, eps, offset=0.0, magnitude=1.0, layout="half"):
    """(dx, dweight) of the above, and what bounds a rounding of each: the sums of the absolute values of its terms."""
    x = np.asarray(x, np.float64)
    g = np.asarray(dy, np.float64) if angles is None else rope(dy, pos, angles, magnitude, layout, inverse=True)
    f = 1.0 if weight is None else offset + np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * r
    dx = r * (g * f - n * (g * f * n).mean(-1, keepdims=True))
    size = r * (np.abs(g * f) + np.abs(n) * np.abs(g * f * n).mean(-1, keepdims=True))
    return dx, (g * n).sum((0, 1)), size, np.abs(g * n).sum((0, 1))


def token_scores(logits, tokens=None, scale=1.0, top=0):
    """(logprob, lse, entropy, top_logprob, top_token) of rows of logits."""
    x = np.asarray(logits, np.float64)
    z = x * scale
    rows, vocab = z.shape
    bad = np.isnan(z).any(-1) | (z == np.inf).any(-1)
    m = np.where(bad, 0.0, z.max(-1))
    none = ~bad & (m == -np.inf)
    m = np.where(none, 0.0, m)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.exp(z - m[:, None])
        lse = m + np.log(e.sum(-1))
        logp = (z - m[:, None]) - np.log(e.sum(-1))[:, None]     # lse may have swallowed the logarithm
        p = np.exp(logp)
        entropy = -np.where(p > 0, p * logp, 0.0).sum(-1)
    lse, entropy = np.where(bad, np.nan, np.where(none, -np.inf, lse)), np.where(bad, np.nan, np.where(none, 0.0, entropy))
    logp = np.where(bad[:, None], np.nan, np.where(none[:, None], -np.inf, logp))
    logprob = None
    if tokens is not None:
        t = np.asarray(tokens)
        here = (t >= 0) & (t < vocab)
        logprob = np.where(here, logp[np.arange(rows), np.where(here, t, 0)], 0.0)
    order = np.argsort(np.where(np.isnan(x), np.inf, -x), axis=-1, kind="stable")
    # of -inf and NaN, both at the end, the numbers come first
    order = np.stack([np.concatenate([o[~np.isnan(r[o])], o[np.isnan(r[o])]]) for o, r in zip(order, x)])[:, :top]
    return logprob, lse, entropy, np.take_along_axis(logp, order, -1), order


def token_scores_backward(logits, tokens, lse, entropy, dlogprob=None, dentropy=None, dlse=None, scale=1.0):
    """dlogits, and the sum of the absolute values of its terms."""
    z = np.asarray(logits, np.float64) * scale
    rows, vocab = z.shape
    col = lambda v: np.zeros((rows, 1)) if v is None else np.asarray(v, np.float64)[:, None]  # noqa: E731
    gp, gh, gl = col(dlogprob), col(dentropy), col(dlse)
    t = np.full(rows, -1) if tokens is None else np.asarray(tokens)
    here = ((t >= 0) & (t < vocab))[:, None]
    gp = np.where(here, gp, 0.0)
    hit = np.arange(vocab)[None] == t[:, None]
    none = np.isneginf(col(lse))
    with np.errstate(invalid="ignore"):
        logp = np.where(none, -np.inf, z - np.where(none, 0.0, col(lse)))
    p = np.exp(logp)
    logp = np.where(p > 0, logp, 0.0)
    h = col(entropy)
    d = gp * (hit & here & ~none) - gp * p - gh * p * (logp + h) + gl * p
    size = np.abs(gp) * (hit & here) + p * (np.abs(gp) + np.abs(gh) * (np.abs(logp) + np.abs(h)) + np.abs(gl))
    return scale * d, scale * size
