"""The serving operators between aq_linear_qkv and the o projection, and after the last layer:
rotary positions, the paged key/value cache (written, quantised, read back), attention of drafted
tokens over that cache, and the verification of the drafts.

``own`` False: plain torch forms in float32. ``own`` True: the library's entry points. Both take the
same prepared state. ``exact`` gives the same outputs from the definitions in float64.
"""
import math

import numpy as np
import torch

own = False

E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100     # smallest stored scale of a quantised vector


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
def listed():
    return [
        # the four query heads of a Gemma-3-1B layer, a few drafted tokens: one launch's latency
        dict(name="rope_step", op="rope", tokens=5, heads=4, dim=256, rot=256, layout="half",
             scaling="none", inverse=False, head_major=False, max_pos=32768),
        # a prefill chunk, part of the head rotated, interleaved pairs, long-context frequencies
        dict(name="rope_prefill", op="rope", tokens=8192, heads=32, dim=128, rot=64, layout="interleaved",
             scaling="yarn", inverse=False, head_major=False, max_pos=131072),
        # the gradient with respect to the input at training length, heads outermost
        dict(name="rope_grad", op="rope", tokens=4099, heads=16, dim=128, rot=128, layout="half",
             scaling="linear", inverse=True, head_major=True, max_pos=16384),
        # one decode step of a Gemma-3-1B layer with a draft of five
        dict(name="kv_step", op="kv", tokens=5, q_heads=4, kv_heads=1, dim=256, page=16, cache="e4m3",
             layout="half", max_pos=32768),
        # a serving batch's chunk, quantised
        dict(name="kv_chunk", op="kv", tokens=8192, q_heads=32, kv_heads=8, dim=128, page=64, cache="e4m3",
             layout="half", max_pos=131072),
        # one token, one sequence, Gemma-3-1B heads, the sliding window of its local layers
        dict(name="attn_token", op="attn", batch=1, tree=1, ctx=1500, q_heads=4, kv_heads=1, dim=256, page=16,
             cache="bf16", window=512, shape="chain", ragged=False),
        # Gemma-3-1B heads, trees of 16 in a small ragged batch, its long layers
        dict(name="attn_tree16", op="attn", batch=8, tree=16, ctx=4001, q_heads=4, kv_heads=1, dim=256, page=32,
             cache="e4m3", window=0, shape="tree", ragged=True),
        # single tokens of a full serving batch: the plain decode step
        dict(name="attn_decode", op="attn", batch=48, tree=1, ctx=6000, q_heads=32, kv_heads=8, dim=128, page=64,
             cache="e4m3", window=0, shape="chain", ragged=True),
        # drafts of eight in a full serving batch
        dict(name="attn_tree8", op="attn", batch=32, tree=8, ctx=8192, q_heads=32, kv_heads=8, dim=128, page=64,
             cache="bf16", window=0, shape="tree", ragged=True),
        # large trees over long contexts
        dict(name="attn_tree64", op="attn", batch=8, tree=64, ctx=32768, q_heads=32, kv_heads=8, dim=128, page=64,
             cache="bf16", window=0, shape="tree", ragged=False),
        # one sequence's draft of five against a 262144-word vocabulary
        dict(name="verify_one", op="verify", batch=1, nodes=5, vocab=262144, dtype="float32", drafts="sampled"),
        # trees drafted from the most likely tokens, a serving batch
        dict(name="verify_trees", op="verify", batch=48, nodes=12, vocab=262144, dtype="bfloat16", drafts="tree"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "kv", "attn", "attn", "verify"])
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        heads = rng.choice([1, 4, 7, 16, 32])
        tokens = min(_log(rng, 1, 16384), (8192 * 32 * 128) // (heads * dim))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, rot=rng.choice([dim, dim // 2, dim // 4]),
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "yarn"]),
                    inverse=rng.random() < 0.4, head_major=rng.random() < 0.4, max_pos=_log(rng, 4096, 1 << 20))
    if op == "kv":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 8])
        group = rng.choice([1, 4, 8])
        tokens = min(_log(rng, 1, 8192), (8192 * 32 * 128) // (kv * group * dim))
        return dict(op=op, tokens=tokens, q_heads=kv * group, kv_heads=kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                    cache=rng.choice(["e4m3", "bf16"]), layout=rng.choice(["half", "interleaved"]),
                    max_pos=_log(rng, 4096, 1 << 20))
    if op == "attn":
        dim = rng.choice([64, 128, 256])
        kv = rng.choice([1, 2, 8])
        group = rng.choice([1, 2, 4, 8])
        tree = _log(rng, 1, 64)
        batch = _log(rng, 1, 48)
        ctx = _log(rng, 3, 32768)
        # no more keys x rows than the largest listed case, and no more cache
        most = (8 * 32768 * 8 * 128) // (kv * dim * batch)
        ctx = max(3, min(ctx, most, (8 * 32768 * 64 * 32 * 128) // (batch * tree * kv * group * dim)))
        return dict(op=op, batch=batch, tree=tree, ctx=ctx, q_heads=kv * group, kv_heads=kv, dim=dim,
                    page=rng.choice([16, 32, 64, 128]), cache=rng.choice(["e4m3", "bf16"]),
                    window=rng.choice([0, 0, 512, 1024]), shape=rng.choice(["tree", "chain"]),
                    ragged=rng.random() < 0.7)
    batch = _log(rng, 1, 48)
    return dict(op=op, batch=batch, nodes=_log(rng, 1, 12), vocab=rng.choice([32000, 50257, 151936, 262144]),
                dtype=rng.choice(["float32", "bfloat16"]), drafts=rng.choice(["sampled", "tree"]))


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _frequencies(rot, scaling, base=10000.0, factor=8.0, original=8192.0):
    """Radians a position for each of rot/2 pairs, and the factor on cos and sin."""
    i = np.arange(rot // 2, dtype=np.float64)
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":   # pairs that turn often keep their frequency, those that hardly turn are interpolated
        dims = [rot * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0)]
        lo, hi = max(math.floor(dims[0]), 0), min(math.ceil(dims[1]), rot - 1)
        ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def _rope_table(rot, scaling, device):
    f, mag = _frequencies(rot, scaling)
    turns = [int(round(float(x) / (2 * math.pi) * 2.0 ** 64)) for x in f]
    return torch.tensor(turns, dtype=torch.int64, device=device), mag


def _lengths(case):
    """Context length of each sequence: the same for all, or spread over [ctx / 8, ctx]."""
    n, ctx = case["batch"], case["ctx"]
    if not case["ragged"] or n == 1:
        return [ctx] * n
    return [max(1, ctx - (ctx * 7 // 8) * ((b * 5) % n) // max(1, n - 1)) for b in range(n)]


def _drafted(case):
    """Drafted tokens of each sequence."""
    n, t = case["batch"], case["tree"]
    return [t - (b % 3 if case["ragged"] and t > 3 else 0) for b in range(n)]


def prepare(case, seed):
    device = "cuda"
    g = _gen(seed, device)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "rope":
        t, h, d = case["tokens"], case["heads"], case["dim"]
        x = torch.randn(h, t, d, generator=g, device=device).to(torch.bfloat16)
        s["x"] = x.transpose(0, 1) if case["head_major"] else x.transpose(0, 1).contiguous()
        s["pos"] = torch.randint(0, case["max_pos"], (t,), generator=g, device=device, dtype=torch.int32)
        s["freq"], s["mag"] = _rope_table(case["rot"], case["scaling"], device)
    elif op == "kv":
        t, hq, hk, d, page = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim", "page"))
        # q, k and v as column slices of one stacked projection output
        qkv = torch.randn(t, (hq + 2 * hk) * d, generator=g, device=device)
        qkv *= torch.exp(0.7 * torch.randn(t, 1, generator=g, device=device))
        qkv = qkv.to(torch.bfloat16)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        s["pos"] = torch.randint(0, case["max_pos"], (t,), generator=g, device=device, dtype=torch.int32)
        s["freq"], s["mag"] = _rope_table(d, "none", device)
        pages = -(-t // page) + 3
        s["slots"] = torch.randperm(pages * page, generator=g, device=device)[:t].contiguous()
        s.update(_empty_cache(pages, case, device))
    elif op == "attn":
        hq, hk, d, page = (case[k] for k in ("q_heads", "kv_heads", "dim", "page"))
        ctx, drafted = _lengths(case), _drafted(case)
        total = sum(drafted)
        s["q"] = (1.5 * torch.randn(total, hq, d, generator=g, device=device)).to(torch.bfloat16)
        need = [-(-(c + n) // page) for c, n in zip(ctx, drafted)]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g, device=device)[:sum(need)].to(torch.int32)
        table = torch.zeros(case["batch"], max(need), dtype=torch.int32, device=device)
        first = 0
        for b, n in enumerate(need):
            table[b, :n] = order[first:first + n]
            first += n
        s["table"] = table
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=device)
        s["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(drafted)]), dtype=torch.int32, device=device)
        s["max_q"], s["scale"] = max(drafted), d ** -0.5
        s.update(_empty_cache(pages, case, device))
        for kv in ("k", "v"):
            for p0 in range(0, pages, 1024):
                p1 = min(pages, p0 + 1024)
                x = torch.randn(p1 - p0, hk, page, d, generator=g, device=device)
                if case["cache"] == "bf16":
                    s[kv + "_cache"][p0:p1] = x.to(torch.bfloat16)
                else:
                    scale = x.abs().amax(-1) * (1.0 / E4M3_MAX)
                    s[kv + "_scale"][p0:p1] = scale
                    s[kv + "_cache"][p0:p1] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        s["mask"] = s["depth"] = None
        if case["shape"] == "tree":
            # each drafted token follows an earlier one or the context; it sees its ancestors and itself
            words = -(-max(drafted) // 64)
            mask = np.zeros((total, words), dtype=np.uint64)
            depth = np.zeros(total, dtype=np.int32)
            r = np.random.RandomState(int(seed) % (2 ** 31))
            at = 0
            for n in drafted:
                for i in range(n):
                    parent = r.randint(-1, i) if i else -1
                    if parent >= 0:
                        mask[at + i] = mask[at + parent]
                        depth[at + i] = depth[at + parent] + 1
                    mask[at + i, i // 64] |= np.uint64(1) << np.uint64(i % 64)
                at += n
            s["mask"] = torch.from_numpy(mask.view(np.int64)).to(device)
            s["depth"] = torch.from_numpy(depth).to(device)
    else:
        b, n, v = case["batch"], case["nodes"], case["vocab"]
        dt = getattr(torch, case["dtype"])
        rows = b * (n + 1)
        p = torch.empty(rows, v, dtype=dt, device=device)
        q = torch.empty(rows, v, dtype=dt, device=device) if case["drafts"] == "sampled" else None
        tokens = torch.empty(b, n, dtype=torch.int32, device=device)
        parent = None
        if case["drafts"] == "tree":
            # one root with three children, each of them with children of its own
            parent = torch.tensor([-1 if i < 3 else (i - 3) // 2 for i in range(n)], dtype=torch.int32,
                                  device=device).repeat(b)
        for j in range(b):
            r0 = j * (n + 1)
            logits = 3.0 * torch.randn(n + 1, v, generator=g, device=device)
            p[r0:r0 + n + 1] = torch.softmax(logits, -1).to(dt)
            if q is not None:
                logits += 0.7 * torch.randn(n + 1, v, generator=g, device=device)
                q[r0:r0 + n + 1] = torch.softmax(logits, -1).to(dt)
                race = torch.empty(n, v, device=device).exponential_(generator=g)
                tokens[j] = (q[r0:r0 + n].float() / race).argmax(-1).to(torch.int32)
            else:
                best = logits.topk(3, -1).indices.to(torch.int32)
                i = torch.arange(n, device=device)
                row = torch.where(i < 3, 0, (i - 3) // 2 + 1)
                tokens[j] = best[row, torch.where(i < 3, i, (i - 3) % 2)]
        s.update(p=p, q=q, tokens=tokens.reshape(-1), parent=parent)
        s["u"] = torch.rand(b * n, generator=g, device=device)
        s["noise"] = torch.empty(b, v, device=device).exponential_(generator=g).clamp_(min=1e-10)
        s["cu"] = torch.arange(0, b * n + 1, n, dtype=torch.int32, device=device)
        s["cap"] = n
    return s


def _empty_cache(pages, case, device):
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    bf16 = case["cache"] == "bf16"
    one = {}
    for kv in ("k", "v"):
        one[kv + "_cache"] = torch.zeros(pages, hk, page, d, dtype=torch.bfloat16 if bf16 else torch.uint8, device=device)
        one[kv + "_scale"] = None if bf16 else torch.ones(pages, hk, page, dtype=torch.float32, device=device)
    return one


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _own_rope, "kv": _own_kv, "attn": _own_attn, "verify": _own_verify}[op](s)
    return {"rope": _plain_rope, "kv": _plain_kv, "attn": _plain_attn, "verify": _plain_verify}[op](s)


def _layout(aq, s):
    return aq.AQ_ROPE_HALF if s["case"]["layout"] == "half" else aq.AQ_ROPE_INTERLEAVED


def _cache(aq, s):
    return aq.KvCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])


def _own_rope(s):
    import rank_weight_reconstruction_gb300 as aq
    rope = aq.Rope(s["freq"], layout=_layout(aq, s), magnitude=s["mag"])
    return {"y": aq.aq_rope(rope, s["pos"], s["x"], inverse=s["case"]["inverse"])}


def _own_kv(s):
    import rank_weight_reconstruction_gb300 as aq
    cache = _cache(aq, s)
    rope = aq.Rope(s["freq"], layout=_layout(aq, s), magnitude=s["mag"])
    q = aq.aq_kv_write(cache, s["k"], s["v"], s["slots"], rope=rope, pos=s["pos"], q=s["q"])
    k, v = aq.aq_kv_read(cache, s["slots"])
    return {"q": q, "k": k, "v": v}


def _own_attn(s):
    import rank_weight_reconstruction_gb300 as aq
    out, lse = aq.aq_tree_attention(_cache(aq, s), s["q"], s["cu"], s["ctx"], s["table"], max_q=s["max_q"],
                                    mask=s["mask"], depth=s["depth"], window=s["case"]["window"], scale=s["scale"],
                                    return_lse=True)
    return {"out": out, "lse": lse}


def _own_verify(s):
    import rank_weight_reconstruction_gb300 as aq
    count, path, token = aq.aq_verify_drafts(s["p"], s["tokens"], s["cu"], s["u"], s["noise"], q=s["q"],
                                             parent=s["parent"], path_cap=s["cap"])
    return {"count": count, "path": path, "token": token}


def _rotate(x, pos, freq, mag, layout, inverse=False):
    """x [T, H, D] in float32 with its first 2 * len(freq) elements rotated."""
    phase = pos.to(torch.int64)[:, None] * freq[None, :]             # fractions of a turn, modulo one turn
    angle = phase.to(torch.float32) * (2.0 ** -64) * (2 * math.pi)
    c, n = torch.cos(angle)[:, None, :] * mag, torch.sin(angle)[:, None, :] * (-mag if inverse else mag)
    half = freq.numel()
    x = x.float()
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_rope(s):
    c = s["case"]
    return {"y": _rotate(s["x"], s["pos"], s["freq"], s["mag"], c["layout"], c["inverse"]).to(torch.bfloat16)}


def _plain_kv(s):
    page = s["case"]["page"]
    q = _rotate(s["q"], s["pos"], s["freq"], s["mag"], s["case"]["layout"]).to(torch.bfloat16)
    k = _rotate(s["k"], s["pos"], s["freq"], s["mag"], s["case"]["layout"])
    at, off = s["slots"] // page, s["slots"] % page
    back = {"q": q}
    back["k"] = _store_and_load(s, "k", k, at, off)
    back["v"] = _store_and_load(s, "v", s["v"].float(), at, off)
    return back


def _store_and_load(s, kv, x, at, off):
    cache, scales = s[kv + "_cache"], s[kv + "_scale"]
    if scales is None:
        cache[at, :, off] = x.to(torch.bfloat16)
        return cache[at, :, off].clone()
    scale = torch.clamp(x.abs().amax(-1) * (1.0 / E4M3_MAX), min=SCALE_FLOOR)
    codes = torch.clamp(x * (1.0 / scale)[..., None], -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    cache[at, :, off] = codes.view(torch.uint8)
    scales[at, :, off] = scale
    return (cache[at, :, off].view(torch.float8_e4m3fn).float() * scales[at, :, off][..., None]).to(torch.bfloat16)


def _visible(s, rows_t, keys, device):
    """[B, T, L]: whether drafted token i of sequence b sees key j of its sequence."""
    ctx, cu, n = s["ctx"].long(), s["cu"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    i = torch.arange(rows_t, device=device)
    j = torch.arange(keys, device=device)
    row = torch.clamp(cu[:-1, None] + i[None, :], max=int(s["q"].size(0)) - 1)          # [B, T]
    inside = j[None, None, :] - ctx[:, None, None]                                       # index among the drafted
    if s["mask"] is None:
        depth = i[None, :].expand(ctx.numel(), -1)
        drafted = inside <= i[None, :, None]
        at = torch.minimum(j[None, :], (ctx + n)[:, None])
    else:
        depth = s["depth"].long()[row]
        idx = torch.clamp(inside, min=0, max=rows_t - 1).expand(-1, rows_t, -1)
        word = torch.gather(s["mask"][row], 2, idx // 64)
        drafted = ((word >> (idx % 64)) & 1).bool()
        key_row = torch.clamp(cu[:-1, None] + torch.clamp(inside[:, 0], min=0), max=int(s["q"].size(0)) - 1)
        at = torch.where(inside[:, 0] < 0, j[None, :], ctx[:, None] + s["depth"].long()[key_row])
    seen = (inside < 0) | (drafted & (inside < n[:, None, None]))
    if s["case"]["window"] > 0:
        seen &= (ctx[:, None] + depth)[:, :, None] - at[:, None, :] < s["case"]["window"]
    return seen & (i[None, :, None] < n[:, None, None])


def _plain_attn(s):
    c = s["case"]
    page, hk, d = c["page"], c["kv_heads"], c["dim"]
    group = c["q_heads"] // hk
    q, table = s["q"], s["table"].long()
    b, keys, t = table.size(0), table.size(1) * page, s["max_q"]
    kv = {}
    for name in ("k", "v"):
        x = s[name + "_cache"][table]                                                    # [B, P, Hk, page, D]
        if s[name + "_scale"] is None:
            x = x.float()
        else:
            x = x.view(torch.float8_e4m3fn).float() * s[name + "_scale"][table][..., None]
        kv[name] = x.transpose(1, 2).reshape(b, hk, keys, d)
    i = torch.arange(t, device=q.device)
    row = torch.clamp(s["cu"].long()[:-1, None] + i[None, :], max=q.size(0) - 1)
    qb = q[row].float().view(b, t, hk, group, d).permute(0, 2, 1, 3, 4).reshape(b, hk, t * group, d)
    seen = _visible(s, t, keys, q.device)[:, None, :, None, :]
    score = torch.matmul(qb, kv["k"].transpose(-1, -2)).view(b, hk, t, group, keys) * s["scale"]
    score = score.masked_fill(~seen, -math.inf)
    m = score.amax(-1, keepdim=True)
    w = torch.exp(score - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = w.sum(-1, keepdim=True)
    out = torch.matmul(w.view(b, hk, t * group, keys), kv["v"]).view(b, hk, t, group, d)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (m + torch.log(total)).squeeze(-1)
    valid = i[None, :] < (s["cu"][1:] - s["cu"][:-1])[:, None]
    out = out.permute(0, 2, 1, 3, 4).reshape(b, t, hk * group, d)[valid]
    lse = lse.permute(0, 2, 1, 3).reshape(b, t, hk * group)[valid]
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _plain_verify(s):
    c = s["case"]
    b, n, v = c["batch"], c["nodes"], c["vocab"]
    p = s["p"].view(b, n + 1, v)
    tok = s["tokens"].long().view(b, n)
    u = s["u"].view(b, n)
    i = torch.arange(n, device=tok.device)
    parent = (s["parent"].long().view(b, n) if s["parent"] is not None else (i - 1).expand(b, n)) + 1    # row of p
    px = p[torch.arange(b, device=tok.device)[:, None], parent, tok].float()
    same = (parent[:, :, None] == parent[:, None, :]) & (i[None, :] < i[:, None])[None]   # an earlier sibling
    if s["q"] is not None:
        qx = s["q"].view(b, n + 1, v)[torch.arange(b, device=tok.device)[:, None], parent, tok].float()
        taken = u * qx < px
    else:
        taken = u * (1.0 - (same * px[:, None, :]).sum(-1)) < px
    first = taken & ~(same & taken[:, None, :]).any(-1)
    # a node is on the path when it and all its ancestors are the first accepted of their siblings: powers of
    # the parent relation up to depth n, by repeated squaring
    up = torch.zeros(b, n + 1, n + 1, device=tok.device)
    up.scatter_(2, torch.cat([torch.zeros_like(parent[:, :1]), parent], 1)[:, :, None], 1.0)
    good = torch.cat([torch.ones_like(first[:, :1]), first], 1).float()
    below = torch.clamp(torch.eye(n + 1, device=tok.device) + up, max=1.0)
    for _ in range(max(1, n.bit_length())):
        below = torch.clamp(torch.matmul(below, below), max=1.0)       # ancestors of each node, itself among them
    path = (torch.matmul(below, (1.0 - good)[:, :, None]).squeeze(-1) == 0)[:, 1:]
    count = path.sum(-1)
    order = torch.where(path, i[None, :], n).sort(-1).values
    nodes = torch.where(order < n, order, -1).to(torch.int32)
    last = torch.where(path, i[None, :] + 1, 0).amax(-1)               # row of p the draw is from
    rows = torch.arange(b, device=tok.device)
    pr = p[rows, last].float()
    tested = parent == last[:, None]
    if s["q"] is not None:
        rest = torch.clamp(pr - s["q"].view(b, n + 1, v)[rows, last].float(), min=0.0)
        weight = torch.where(tested.any(-1)[:, None], rest, pr)
    else:
        gone = torch.zeros(b, v, device=tok.device).scatter_add_(1, tok, tested.float())
        weight = torch.where(gone > 0, torch.zeros_like(pr), pr)
    weight = torch.where((weight > 0).any(-1, keepdim=True), weight, pr)
    score = weight / s["noise"]
    best = score.amax(-1, keepdim=True)
    j = torch.arange(v, device=tok.device)
    token = torch.where(score == best, j[None, :], v).amin(-1)
    return {"count": count.to(torch.int32), "path": nodes, "token": token.to(torch.int32)}


# --------------------------------------------------------------------------------------
# work and exact values
# --------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "rope":
        n = case["tokens"] * case["heads"] * case["dim"]
        return {"bytes": 4 * n + 4 * case["tokens"], "flops": 3 * case["tokens"] * case["heads"] * case["rot"]}
    if op == "kv":
        t, d, hk = case["tokens"], case["dim"], case["kv_heads"]
        cell = 2 * d if case["cache"] == "bf16" else d + 4
        per = case["q_heads"] * d * 4 + 2 * hk * (2 * d + cell)        # the write
        per += 2 * hk * (cell + 2 * d) + 20                            # the read, positions and slots
        return {"bytes": t * per, "flops": 3 * t * d * (case["q_heads"] + hk)}
    if op == "attn":
        d, hk, hq = case["dim"], case["kv_heads"], case["q_heads"]
        cell = 2 * d if case["cache"] == "bf16" else d + 4
        total, moved = 0, 0
        for c, n in zip(_lengths(case), _drafted(case)):
            seen = c if case["window"] <= 0 else min(c, case["window"] - 1)
            total += n * seen + n * (n + 1) // 2
            moved += (seen + n) * hk * cell * 2 + n * hq * (4 * d + 4)
        return {"bytes": moved, "flops": 4 * total * hq * d}
    size = 4 if case["dtype"] == "float32" else 2
    rows = 2 if case["drafts"] == "sampled" else 1
    return {"bytes": case["batch"] * case["vocab"] * (size * rows + 4), "flops": case["batch"] * case["vocab"] * rows}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return {"y": _exact_rope(s["x"].double(), s["pos"], case["rot"], case["scaling"], case["layout"],
                                 -1.0 if case["inverse"] else 1.0)}
    if op == "kv":
        d = case["dim"]
        out = {"q": _exact_rope(s["q"].double(), s["pos"], d, "none", case["layout"], 1.0)}
        for name in ("k", "v"):
            x = s[name].double()
            if name == "k":
                x = _exact_rope(x, s["pos"], d, "none", case["layout"], 1.0)
            if case["cache"] == "e4m3":
                step = (x.abs().max(-1, keepdim=True).values / 448).clamp_min(SCALE_FLOOR)
                x = _nearest_e4m3(x / step) * step
            out[name] = x
        return out
    if op == "attn":
        if work(case)["flops"] > 4e12:
            return None
        return _exact_attn(s, case)
    return _exact_verify(s, case)


def _exact_rope(x, pos, rot, scaling, layout, sign):
    f, mag = _frequencies(rot, scaling)
    a = pos.double()[:, None] * torch.from_numpy(f).to(x.device)[None]
    z = torch.polar(torch.full_like(a, mag), sign * a)[:, None, :]
    y = x.clone()
    if layout == "half":
        w = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * z
        y[..., :rot // 2], y[..., rot // 2:rot] = w.real, w.imag
    else:
        w = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * z
        y[..., 0:rot:2], y[..., 1:rot:2] = w.real, w.imag
    return y


def _nearest_e4m3(x):
    """Nearest E4M3 value, ties to even, by the spacing of the format at |x|."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_attn(s, case):
    hk, d, page, w = case["kv_heads"], case["dim"], case["page"], case["window"]
    group = case["q_heads"] // hk
    outs, lses, at = [], [], 0
    for b, (c, n) in enumerate(zip(_lengths(case), _drafted(case))):
        pages = s["table"][b, :-(-(c + n) // page)].long()
        kv = []
        for name in ("k", "v"):
            x = s[name + "_cache"][pages]
            x = x.double() if s[name + "_scale"] is None else (
                x.view(torch.float8_e4m3fn).double() * s[name + "_scale"][pages].double()[..., None])
            kv.append(x.permute(1, 0, 2, 3).flatten(1, 2)[:, :c + n])
        see = torch.ones(n, c + n, dtype=torch.bool, device=s["q"].device)
        depth = torch.arange(n, device=s["q"].device)
        see[:, c:] = depth[:, None] >= depth[None, :]
        if s["mask"] is not None:
            depth = s["depth"][at:at + n].long()
            see[:, c:] = ((s["mask"][at:at + n].repeat_interleave(64, 1)
                           >> torch.arange(64, device=depth.device).repeat(s["mask"].size(1))) & 1).bool()[:, :n]
        if w > 0:
            where = torch.cat([torch.arange(c, device=depth.device), c + depth])
            see &= (c + depth)[:, None] - where[None, :] < w
        q = s["q"][at:at + n].double()
        out = torch.empty(n, hk * group, d, dtype=torch.float64, device=q.device)
        lse = torch.empty(n, hk * group, dtype=torch.float64, device=q.device)
        for h in range(hk * group):
            sc = (q[:, h] @ kv[0][h // group].T) * d ** -0.5
            sc[~see] = -math.inf
            lse[:, h] = torch.logsumexp(sc, -1)
            out[:, h] = torch.nan_to_num(torch.exp(sc - lse[:, h:h + 1])) @ kv[1][h // group]
        outs.append(out)
        lses.append(lse)
        at += n
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_verify(s, case):
    n, v = case["nodes"], case["vocab"]
    counts, paths, draws = [], [], []
    for b in range(case["batch"]):
        tok, u = s["tokens"][b * n:(b + 1) * n].tolist(), s["u"][b * n:(b + 1) * n].double().tolist()
        parent = list(range(-1, n - 1)) if s["parent"] is None else s["parent"][b * n:(b + 1) * n].tolist()
        here, path = -1, []
        while True:
            row = b * (n + 1) + here + 1
            p = s["p"][row].double()
            left = p.clone()
            mass, chosen = 1.0, None
            for i in [i for i in range(n) if parent[i] == here]:
                if s["q"] is not None:
                    q = s["q"][row].double()
                    if u[i] * float(q[tok[i]]) < float(left[tok[i]]):
                        chosen = i
                        break
                    left = (left - q).clamp_min(0)
                    total = float(left.sum())
                    left = left / total if total > 0 else left
                else:
                    if u[i] * mass < float(left[tok[i]]):
                        chosen = i
                        break
                    mass -= float(left[tok[i]])
                    left[tok[i]] = 0
            if chosen is None:
                break
            path.append(chosen)
            here = chosen
        if float(left.sum()) <= 0:
            left = p
        draws.append(int((left / s["noise"][b].double()).argmax()))
        counts.append(len(path))
        paths.append(path + [-1] * (n - len(path)))
    as_int = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"count": as_int(counts), "path": as_int(paths), "token": as_int(draws)}
