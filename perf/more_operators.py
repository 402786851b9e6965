"""Operators around a decode step on quantised weights: products with the 4-bit weights that the
precompute makes, norms of the query and key heads with the rotation (with their gradient, and on the
way into the cache), and the scores of tokens from the logits (with their gradient).

``own`` False: plain torch forms in float32. ``own`` True: the library's entry points. Both take the
same prepared state. ``exact`` gives the same outputs from the definitions in float64.
"""
import math

import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
E4M3_MAX = 448.0
SCALE_FLOOR = 2.0 ** -100     # smallest stored scale of a quantised vector of the cache


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
def listed():
    return [
        # q, k and v of a Gemma-3-1B layer for one token, in one call: a call's latency
        dict(name="nvfp4_qkv_step", op="nvfp4", outs="1024,256,256", inp=1152, tokens=1, layout="linear"),
        # its down projection for a batch of 16, scales as the block-scaled matrix instructions read them
        dict(name="nvfp4_down_16", op="nvfp4", outs="1152", inp=6912, tokens=16, layout="128x4"),
        # a 31B-class projection for a tree of eight drafted tokens
        dict(name="nvfp4_31b_8", op="nvfp4", outs="21504", inp=5376, tokens=8, layout="linear"),
        # the output head over Gemma's vocabulary for a few drafted tokens
        dict(name="nvfp4_head_5", op="nvfp4", outs="262144", inp=1152, tokens=5, layout="128x4"),
        # a draft of five tokens of a Gemma-3-1B layer: a call's latency
        dict(name="norm_step", op="norm", tokens=5, q_heads=4, kv_heads=1, dim=256, rot=256, layout="half",
             head_major=False, max_pos=32768),
        # a prefill chunk on its way into the cache, quantised, and read back
        dict(name="norm_cache_chunk", op="norm_kv", tokens=8192, q_heads=32, kv_heads=8, dim=128, rot=128, page=64,
             cache="e4m3", layout="half", max_pos=131072),
        # the same norms where a training step has them: forward at an odd length, part of the head turned
        dict(name="norm_train", op="norm", tokens=16385, q_heads=16, kv_heads=4, dim=128, rot=64, layout="interleaved",
             head_major=False, max_pos=16384),
        # and backward, heads outermost, with the gradients of both weights
        dict(name="norm_grad", op="norm_grad", tokens=8195, q_heads=32, kv_heads=8, dim=128, rot=128, layout="half",
             head_major=True, max_pos=16384),
        # what a serving step reports for a draft of five: the drafts' log probabilities and five alternatives
        dict(name="scores_step", op="scores", rows=5, vocab=262144, dtype="bfloat16", top=5, scale=1.0),
        # an odd vocabulary in float32 at a temperature, 20 alternatives
        dict(name="scores_odd", op="scores", rows=333, vocab=50257, dtype="float32", top=20, scale=1.25),
        # scoring a text: 1024 rows, nothing but log probabilities and entropies
        dict(name="scores_text", op="scores", rows=1024, vocab=262144, dtype="bfloat16", top=0, scale=1.0),
        # the loss's gradient over the same text
        dict(name="scores_grad", op="scores_grad", rows=1024, vocab=262144, dtype="bfloat16", top=0, scale=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["nvfp4", "nvfp4", "norm", "norm_kv", "norm_grad", "scores", "scores", "scores_grad"])
    if op == "nvfp4":
        inp = 16 * _log(rng, 4, 1344)
        most = (262144 * 1152) // inp
        n = rng.choice([1, 1, 1, 2, 3])
        outs = [_log(rng, 64, min(262144, most // n)) for _ in range(n)]
        return dict(op=op, outs=",".join(map(str, outs)), inp=inp, tokens=_log(rng, 1, 32),
                    layout=rng.choice(["linear", "128x4"]))
    if op in ("norm", "norm_kv", "norm_grad"):
        dim = rng.choice([64, 80, 128, 256])
        kv = rng.choice([1, 2, 8])
        hq = kv * rng.choice([1, 4, 5])
        tokens = min(_log(rng, 1, 32768), (8192 * 40 * 128) // ((hq + kv) * dim))
        c = dict(op=op, tokens=tokens, q_heads=hq, kv_heads=kv, dim=dim, rot=rng.choice([dim, dim, dim // 32 * 16]),
                 layout=rng.choice(["half", "interleaved"]), max_pos=_log(rng, 4096, 1 << 20))
        if op == "norm_kv":
            c.update(page=rng.choice([16, 32, 64, 128]), cache=rng.choice(["e4m3", "bf16"]))
        else:
            c["head_major"] = rng.random() < 0.4
        return c
    vocab = rng.choice([32000, 50257, 151936, 262144, _log(rng, 1000, 262144)])
    dtype = rng.choice(["float32", "bfloat16"])
    size = 4 if dtype == "float32" else 2
    return dict(op=op, rows=min(_log(rng, 1, 4096), (1024 * 262144 * 2) // (vocab * size)), vocab=vocab, dtype=dtype,
                top=rng.choice([0, 1, 5, 20, 32]) if op == "scores" else 0, scale=rng.choice([1.0, 1.25, 0.5]))


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _outs(case):
    return [int(x) for x in case["outs"].split(",")]


def _scale_bytes(scales, layout):
    """E4M3 scales [out, in/16] as the given layout holds them."""
    if layout == "linear":
        return scales
    out, cols = scales.shape
    pad = torch.zeros(-(-out // 128) * 128, -(-cols // 4) * 4, dtype=torch.uint8, device=scales.device)
    pad[:out, :cols] = scales
    # tiles of 128 rows by 4 columns, one after another along the row band: row r, column k at 16 (r % 32) + 4 (r // 32) + k
    return pad.view(-1, 4, 32, pad.size(1) // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _quantised_weight(g, out, inp, layout, device):
    """Gaussian rows of differing size, quantised the way the precompute quantises."""
    sigma = inp ** -0.5
    gscale = torch.tensor([6.0 * sigma / (6 * E4M3_MAX)], dtype=torch.float32, device=device)
    q = torch.empty(out, inp // 2, dtype=torch.uint8, device=device)
    sf = torch.empty(out, inp // 16, dtype=torch.uint8, device=device)
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=device)
    for r0 in range(0, out, 16384):
        r1 = min(out, r0 + 16384)
        w = torch.randn(r1 - r0, inp // 16, 16, generator=g, device=device) * sigma
        w *= torch.exp(0.3 * torch.randn(r1 - r0, 1, 1, generator=g, device=device))
        s = (w.abs().amax(-1) / (6 * gscale)).clamp(max=E4M3_MAX).to(torch.float8_e4m3fn)
        sf[r0:r1] = s.view(torch.uint8)
        w /= (s.float() * gscale).clamp(min=1e-30)[..., None]
        code = torch.bucketize(w.abs(), edges) + 8 * (w < 0)
        code = code.view(r1 - r0, inp // 2, 2).to(torch.uint8)
        q[r0:r1] = code[..., 0] | (code[..., 1] << 4)
    return q, _scale_bytes(sf, layout).contiguous(), gscale


def _rope_table(rot, device, base=10000.0):
    turns = [int(round(base ** (-2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64)) for i in range(rot // 2)]
    return torch.tensor(turns, dtype=torch.int64, device=device)


def prepare(case, seed):
    device = "cuda"
    g = _gen(seed, device)
    op = case["op"]
    s = {"case": dict(case)}
    if op == "nvfp4":
        inp, m = case["inp"], case["tokens"]
        x = torch.randn(m, inp, generator=g, device=device) * torch.exp(torch.randn(m, 1, generator=g, device=device))
        # a few channels many times larger than the rest, as activations have them
        x *= torch.where(torch.rand(inp, generator=g, device=device) < 0.005, 20.0, 1.0)
        s["x"] = x.to(torch.bfloat16)
        s["w"] = [_quantised_weight(g, out, inp, case["layout"], device) for out in _outs(case)]
        return s
    if op.startswith("norm"):
        t, hq, hk, d = (case[k] for k in ("tokens", "q_heads", "kv_heads", "dim"))
        # q, k and v as column slices of one stacked projection output, or tensors with heads outermost
        qkv = torch.randn(t, (hq + 2 * hk) * d, generator=g, device=device)
        qkv *= torch.exp(0.7 * torch.randn(t, 1, generator=g, device=device))
        qkv = qkv.to(torch.bfloat16)
        cut = {"q": qkv[:, :hq * d].unflatten(1, (hq, d)), "k": qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d)),
               "v": qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))}
        major = case.get("head_major", False)
        own_heads = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1) if major else x  # noqa: E731
        s["q"], s["k"], s["v"] = own_heads(cut["q"]), own_heads(cut["k"]), cut["v"]
        s["q_weight"] = (0.3 * torch.randn(d, generator=g, device=device)).to(torch.bfloat16)
        s["k_weight"] = (0.3 * torch.randn(d, generator=g, device=device)).to(torch.bfloat16)
        s["eps"], s["offset"] = 1e-6, 1.0
        s["pos"] = torch.randint(0, case["max_pos"], (t,), generator=g, device=device, dtype=torch.int32)
        s["freq"] = _rope_table(case["rot"], device)
        if op == "norm_grad":
            for name, h in (("dq_out", hq), ("dk_out", hk)):
                shape = (h, t, d) if major else (t, h, d)
                dy = torch.randn(shape, generator=g, device=device).to(torch.bfloat16)
                s[name] = dy.transpose(0, 1) if major else dy
        if op == "norm_kv":
            page = case["page"]
            pages = -(-t // page) + 3
            s["slots"] = torch.randperm(pages * page, generator=g, device=device)[:t].contiguous()
            bf16 = case["cache"] == "bf16"
            for kv in ("k", "v"):
                s[kv + "_cache"] = torch.zeros(pages, hk, page, d, dtype=torch.bfloat16 if bf16 else torch.uint8, device=device)
                s[kv + "_scale"] = None if bf16 else torch.ones(pages, hk, page, dtype=torch.float32, device=device)
        return s
    rows, v = case["rows"], case["vocab"]
    dt = getattr(torch, case["dtype"])
    logits = torch.empty(rows, v, dtype=dt, device=device)
    tokens = torch.empty(rows, dtype=torch.int32, device=device)
    lse, entropy = torch.empty(rows, device=device), torch.empty(rows, device=device)
    step = max(1, (1 << 26) // v)
    for r0 in range(0, rows, step):
        r1 = min(rows, r0 + step)
        z = 2.5 * torch.randn(r1 - r0, v, generator=g, device=device)
        z += 6.0 * (torch.rand(r1 - r0, v, generator=g, device=device) < 20.0 / v)      # a few likely words
        logits[r0:r1] = z.to(dt)
        z = logits[r0:r1].float() * case["scale"]
        # a word drawn from the model's own law
        race = torch.empty(r1 - r0, v, device=device).exponential_(generator=g)
        tokens[r0:r1] = (z - race.log()).argmax(-1).to(torch.int32)
        if op == "scores_grad":     # what the forward call left
            z = z.double()
            lse[r0:r1] = torch.logsumexp(z, -1).float()
            p = torch.softmax(z, -1)
            entropy[r0:r1] = -(p * torch.log(p.clamp_min(1e-300))).sum(-1).float()
    if rows > 16:                   # places without a token, as a padded batch has them
        tokens[torch.rand(rows, generator=g, device=device) < 0.05] = -1
    s.update(logits=logits, tokens=tokens)
    if op == "scores_grad":
        s["lse"], s["entropy"] = lse, entropy
        s["dlogprob"] = -torch.rand(rows, generator=g, device=device) / rows
        s["dentropy"] = torch.full((rows,), -0.01 / rows, device=device)
    return s


# --------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return {"nvfp4": _own_nvfp4, "norm": _own_norm, "norm_kv": _own_norm_kv, "norm_grad": _own_norm_grad,
                "scores": _own_scores, "scores_grad": _own_scores_grad}[op](s)
    return {"nvfp4": _plain_nvfp4, "norm": _plain_norm, "norm_kv": _plain_norm_kv, "norm_grad": _plain_norm_grad,
            "scores": _plain_scores, "scores_grad": _plain_scores_grad}[op](s)


def _own_nvfp4(s):
    import rank_weight_reconstruction_gb300 as aq
    layout = aq.AQ_SF_LINEAR if s["case"]["layout"] == "linear" else aq.AQ_SF_128X4
    return aq.aq_nvfp4_linear_multi([aq.Nvfp4Weight(q, sf, g, layout) for q, sf, g in s["w"]], s["x"])


def _norms(aq, s):
    rope = aq.Rope(s["freq"], layout=aq.AQ_ROPE_HALF if s["case"]["layout"] == "half" else aq.AQ_ROPE_INTERLEAVED)
    return (aq.HeadNorm(s["q_weight"], eps=s["eps"], offset=s["offset"]),
            aq.HeadNorm(s["k_weight"], eps=s["eps"], offset=s["offset"]), rope)


def _own_norm(s):
    import rank_weight_reconstruction_gb300 as aq
    qn, kn, rope = _norms(aq, s)
    q, k = aq.aq_qk_norm_rope(s["q"], s["k"], qn, kn, rope=rope, pos=s["pos"])
    return {"q": q, "k": k}


def _own_norm_kv(s):
    import rank_weight_reconstruction_gb300 as aq
    qn, kn, rope = _norms(aq, s)
    cache = aq.KvCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    q = aq.aq_kv_write(cache, s["k"], s["v"], s["slots"], rope=rope, pos=s["pos"], q=s["q"], q_norm=qn, k_norm=kn)
    k, v = aq.aq_kv_read(cache, s["slots"])
    return {"q": q, "k": k, "v": v}


def _own_norm_grad(s):
    import rank_weight_reconstruction_gb300 as aq
    qn, kn, rope = _norms(aq, s)
    dq, dk, dqw, dkw = aq.aq_qk_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], qn, kn, rope=rope, pos=s["pos"])
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _own_scores(s):
    import rank_weight_reconstruction_gb300 as aq
    r = aq.aq_token_logprobs(s["logits"], s["tokens"], scale=s["case"]["scale"], top=s["case"]["top"])
    out = {"logprob": r.logprob, "lse": r.lse, "entropy": r.entropy}
    return {**out, "top_logprob": r.top_logprob, "top_token": r.top_token} if s["case"]["top"] else out


def _own_scores_grad(s):
    import rank_weight_reconstruction_gb300 as aq
    return {"dlogits": aq.aq_token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"], s["dlogprob"],
                                                     dentropy=s["dentropy"], scale=s["case"]["scale"])}


def _plain_weight(q, sf, layout, inp):
    """The values that the codes and block scales stand for, float32 [out, in]."""
    table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float32, device=q.device)
    v = torch.stack([table[(q & 15).long()], table[(q >> 4).long()]], -1).view(q.size(0), inp // 16, 16)
    if layout != "linear":
        r = torch.arange(q.size(0), device=q.device)[:, None]
        k = torch.arange(inp // 16, device=q.device)[None, :]
        at = ((r // 128) * (-(-(inp // 16) // 4)) + k // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + k % 4
        sf = sf[at]
    return (v * sf.view(torch.float8_e4m3fn).float()[..., None]).view(q.size(0), inp)


def _plain_nvfp4(s):
    c, x = s["case"], s["x"].float()
    return [(torch.matmul(x, _plain_weight(q, sf, c["layout"], c["inp"]).T) * g).to(torch.bfloat16) for q, sf, g in s["w"]]


def _turn(x, pos, freq, layout, inverse=False):
    """x [T, H, D] in float32 with its first 2 * len(freq) elements rotated."""
    phase = pos.to(torch.int64)[:, None] * freq[None, :]             # fractions of a turn, modulo one turn
    angle = phase.to(torch.float32) * (2.0 ** -64) * (2 * math.pi)
    c, n = torch.cos(angle)[:, None, :], torch.sin(angle)[:, None, :] * (-1.0 if inverse else 1.0)
    half = freq.numel()
    if layout == "half":
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _plain_head(s, name):
    x = s[name].float()
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    return _turn(n * (s["offset"] + s[name + "_weight"].float()), s["pos"], s["freq"], s["case"]["layout"])


def _plain_norm(s):
    return {"q": _plain_head(s, "q").to(torch.bfloat16), "k": _plain_head(s, "k").to(torch.bfloat16)}


def _plain_norm_kv(s):
    page = s["case"]["page"]
    q = _plain_head(s, "q").to(torch.bfloat16)
    at = (s["slots"] // page, slice(None), s["slots"] % page)
    back = {name: _plain_cell(s, name, x, at) for name, x in (("k", _plain_head(s, "k")), ("v", s["v"].float()))}
    return {"q": q, **back}


def _plain_cell(s, name, x, at):
    """x [T, heads, dim] into the cache and out again."""
    if s["case"]["cache"] == "bf16":
        s[name + "_cache"][at] = x.to(torch.bfloat16)
        return s[name + "_cache"][at]
    scale = (x.abs().amax(-1) * (1.0 / E4M3_MAX)).clamp_min(SCALE_FLOOR)
    codes = (x * (1.0 / scale)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    s[name + "_cache"][at], s[name + "_scale"][at] = codes, scale
    held = s[name + "_cache"][at].view(torch.float8_e4m3fn).float()
    return (held * s[name + "_scale"][at][..., None]).to(torch.bfloat16)


def _plain_norm_grad(s):
    dq, dqw = _plain_head_grad(s, "q")
    dk, dkw = _plain_head_grad(s, "k")
    return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}


def _plain_head_grad(s, name):
    x = s[name].float()
    dy = _turn(s["d" + name + "_out"].float(), s["pos"], s["freq"], s["case"]["layout"], inverse=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"])
    n = x * r
    dn = dy * (s["offset"] + s[name + "_weight"].float())
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    # sums over all tokens and heads: in 64 bits
    return dx.to(torch.bfloat16), (dy * n).sum((0, 1), dtype=torch.float64).float()


def _plain_scores(s):
    c = s["case"]
    z = s["logits"].float() * c["scale"]
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(-1, keepdim=True)
    lse = top + torch.log(total)
    entropy = torch.log(total[:, 0]) - (e * (z - top)).sum(-1) / total[:, 0]
    t = s["tokens"].long()
    logprob = torch.where(t >= 0, z.gather(1, t.clamp_min(0)[:, None])[:, 0] - lse[:, 0], torch.zeros_like(lse[:, 0]))
    out = {"logprob": logprob, "lse": lse[:, 0], "entropy": entropy}
    if c["top"]:
        # one whole number a word: its logit's order, and of equal ones the lowest index first
        bits = (s["logits"].float() + 0.0).view(torch.int32).to(torch.int64)
        key = torch.where(bits < 0, bits ^ 0x7fffffff, bits) * (1 << 32) + ((1 << 32) - 1 - torch.arange(c["vocab"], device=z.device))
        key = key.topk(c["top"], -1).values
        word = (1 << 32) - 1 - (key & 0xffffffff)
        out["top_logprob"], out["top_token"] = z.gather(1, word) - lse, word.to(torch.int32)
    return out


def _plain_scores_grad(s):
    scale = s["case"]["scale"]
    logp = s["logits"].float() * scale - s["lse"][:, None]
    t = s["tokens"].long()
    g = torch.where(t >= 0, s["dlogprob"], torch.zeros_like(s["dlogprob"]))[:, None]
    d = torch.exp(logp) * (-g - s["dentropy"][:, None] * (logp + s["entropy"][:, None]))
    d.scatter_add_(1, t.clamp_min(0)[:, None], g)
    return {"dlogits": (d * scale).to(s["logits"].dtype)}


# --------------------------------------------------------------------------------------
# work and exact values
# --------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "nvfp4":
        out, inp, m = sum(_outs(case)), case["inp"], case["tokens"]
        return {"bytes": out * inp // 2 + out * inp // 16 + 2 * m * (inp + out), "flops": 2 * m * out * inp}
    if op.startswith("norm"):
        t, d, hq, hk = (case[k] for k in ("tokens", "dim", "q_heads", "kv_heads"))
        n = t * (hq + hk) * d
        if op == "norm":
            return {"bytes": 4 * n + 4 * t, "flops": 8 * n}
        if op == "norm_grad":
            return {"bytes": 6 * n + 4 * t + 12 * d, "flops": 16 * n}
        cell = 2 * d if case["cache"] == "bf16" else d + 4
        # the write, and the read back
        return {"bytes": t * (4 * hq * d + 2 * hk * (2 * d + cell) + 2 * hk * (cell + 2 * d) + 20), "flops": 8 * n}
    n = case["rows"] * case["vocab"]
    size = 4 if case["dtype"] == "float32" else 2
    if op == "scores":
        return {"bytes": n * size + case["rows"] * (16 + 8 * case["top"]), "flops": 6 * n}
    return {"bytes": 2 * n * size + 20 * case["rows"], "flops": 8 * n}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "nvfp4":
        return [_exact_product(s["x"].double(), q, sf, g, case) for q, sf, g in s["w"]]
    if op == "norm":
        return {name: _exact_head(s, name)[0] for name in ("q", "k")}
    if op == "norm_kv":
        held = {"k": _exact_head(s, "k")[0], "v": s["v"].double()}
        if case["cache"] == "e4m3":
            for name, x in held.items():
                step = (x.abs().max(-1, keepdim=True).values / 448).clamp_min(SCALE_FLOOR)
                held[name] = _nearest_e4m3(x / step) * step
        return {"q": _exact_head(s, "q")[0], **held}
    if op == "norm_grad":
        out = {}
        for name in ("q", "k"):
            with torch.enable_grad():
                y, x, w = _exact_head(s, name, leaves=True)
                dx, dw = torch.autograd.grad(y, (x, w), s["d" + name + "_out"].double())
            out["d" + name], out["d" + name + "_weight"] = dx, dw
        return out
    return _exact_scores(s, case)


def _exact_product(x, q, sf, g, case):
    inp, out = case["inp"], q.size(0)
    y = torch.empty(x.size(0), out, dtype=torch.float64, device=x.device)
    if case["layout"] != "linear":
        # undo the tiles: [bands, column tiles, 32, 4, 4] -> rows by columns
        sf = sf.view(-(-out // 128), -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-(-out // 128) * 128, -1)[:out, :inp // 16]
    for r0 in range(0, out, 8192):
        code = q[r0:r0 + 8192].to(torch.int64)
        code = torch.stack([code % 16, code // 16], -1).flatten(1)
        mag, sign = code % 8, 1.0 - 2.0 * (code // 8)
        # one bit of fraction: mag / 2 below 2, then (2 + bit) * 2^(exponent - 2)
        val = torch.where(mag < 2, mag * 0.5, (2.0 + mag % 2) * torch.exp2((mag // 2 - 2).double()))
        w = val * sign * sf[r0:r0 + 8192].view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
        y[:, r0:r0 + 8192] = x @ w.T
    return y * g.double()


def _exact_head(s, name, leaves=False):
    x, w = s[name].double(), s[name + "_weight"].double()
    if leaves:
        x, w = x.detach().requires_grad_(), w.detach().requires_grad_()
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * (s["offset"] + w)
    rot = s["case"]["rot"]
    f = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device=x.device)
    a = s["pos"].double()[:, None] * f[None]
    z = torch.polar(torch.ones_like(a), a)[:, None, :]
    if s["case"]["layout"] == "half":
        t = torch.complex(n[..., :rot // 2], n[..., rot // 2:rot]) * z
        y = torch.cat([t.real, t.imag, n[..., rot:]], -1)
    else:
        t = torch.complex(n[..., 0:rot:2], n[..., 1:rot:2]) * z
        y = torch.cat([torch.view_as_real(t).flatten(-2), n[..., rot:]], -1)
    return y, x, w


def _nearest_e4m3(x):
    """Nearest E4M3 value, ties to even, by the spacing of the format at |x|."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -6))).clamp(-6, 8)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_scores(s, case):
    rows, v, scale, top = case["rows"], case["vocab"], case["scale"], case["top"]
    parts = []
    step = max(1, (1 << 25) // v)
    for r0 in range(0, rows, step):
        at = slice(r0, min(rows, r0 + step))
        x = s["logits"][at].double()
        logp = torch.log_softmax(x * scale, -1)
        p = torch.exp(logp)
        tok = s["tokens"][at].long()
        entropy = -(p * logp).sum(-1)
        if case["op"] == "scores":
            one = {"logprob": torch.where(tok >= 0, logp.gather(1, tok.clamp_min(0)[:, None])[:, 0], 0.0),
                   "lse": torch.logsumexp(x * scale, -1), "entropy": entropy}
            if top:
                word = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
                one["top_logprob"], one["top_token"] = logp.gather(1, word), word.to(torch.int32)
        else:
            g = torch.where(tok >= 0, s["dlogprob"][at].double(), 0.0)[:, None]
            hit = torch.arange(v, device=x.device)[None] == tok[:, None]
            d = g * (hit.double() - p) - s["dentropy"][at].double()[:, None] * p * (logp + entropy[:, None])
            one = {"dlogits": d * scale}
        parts.append(one)
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}
