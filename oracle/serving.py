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
