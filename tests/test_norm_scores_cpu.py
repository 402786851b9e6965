"""Refusals of the calls around a decode step on quantised weights: head norms, NVFP4 products, token scores. The checks run on the
host before any device work, so placeholder pointers are never dereferenced."""
import ctypes

import pytest

import rank_weight_reconstruction_gb300 as aq
from rank_weight_reconstruction_gb300 import binding as b, build_lib

A, B, C, D_, E, F = (i << 28 for i in range(1, 7))


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return b.load()


def ref(x):
    return None if x is None else ctypes.byref(x)


# ---- head norms ----
def heads(data=A, tok=256, head=64, n=4):
    return b.c_heads(data, tok, head, n)


def norm(weight=0x1000, eps=1e-6, offset=1.0):
    return b.c_head_norm(weight, eps, offset)


ROPE = b.c_rope(0x2000, 64, 0, 1.0)


def call_norm(lib, qn=norm(), kn=norm(), rope=ROPE, pos=0x3000, T=5, dim=64, q=heads(), qo=heads(B), k=heads(C, 128, 64, 2), ko=heads(D_, 128, 64, 2)):
    return lib.aq_qk_norm_rope(ref(qn), ref(kn), ref(rope), pos, T, dim, ref(q), ref(qo), ref(k), ref(ko), None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), b.AQ_ERR_SHAPE), (dict(dim=72), b.AQ_ERR_SHAPE), (dict(dim=272), b.AQ_ERR_SHAPE), (dict(q=None), b.AQ_ERR_INVALID_ARG),
    (dict(qo=None), b.AQ_ERR_INVALID_ARG), (dict(ko=None), b.AQ_ERR_INVALID_ARG), (dict(k=None, ko=None), b.AQ_ERR_INVALID_ARG),
    (dict(pos=None), b.AQ_ERR_INVALID_ARG), (dict(rope=b.c_rope(0x2000, 24, 0, 1.0)), b.AQ_ERR_SHAPE),
    (dict(rope=b.c_rope(0x2000, 128, 0, 1.0)), b.AQ_ERR_SHAPE), (dict(qn=norm(eps=0.0)), b.AQ_ERR_INVALID_ARG),
    (dict(qn=norm(eps=float("nan"))), b.AQ_ERR_INVALID_ARG), (dict(kn=norm(eps=float("inf"))), b.AQ_ERR_INVALID_ARG),
    (dict(kn=norm(offset=float("inf"))), b.AQ_ERR_INVALID_ARG), (dict(kn=norm(weight=0x1008)), b.AQ_ERR_ALIGNMENT),
    (dict(qo=heads(B, n=3)), b.AQ_ERR_SHAPE), (dict(q=heads(n=0), qo=heads(B, n=0)), b.AQ_ERR_SHAPE), (dict(q=heads(A + 8)), b.AQ_ERR_ALIGNMENT),
    (dict(q=heads(tok=260)), b.AQ_ERR_ALIGNMENT), (dict(q=heads(head=32)), b.AQ_ERR_SHAPE), (dict(qo=heads(B, tok=64)), b.AQ_ERR_SHAPE),
    (dict(qo=heads(A + 128)), b.AQ_ERR_OVERLAP), (dict(qo=heads(A, tok=512)), b.AQ_ERR_OVERLAP), (dict(ko=heads(A, 128, 64, 2)), b.AQ_ERR_OVERLAP),
    (dict(ko=heads(B + 64, 128, 64, 2)), b.AQ_ERR_OVERLAP), (dict(qn=norm(weight=B + 256)), b.AQ_ERR_OVERLAP), (dict(pos=B + 64), b.AQ_ERR_OVERLAP),
    (dict(rope=b.c_rope(D_ + 64, 64, 0, 1.0)), b.AQ_ERR_OVERLAP),
])
def test_norm_refusals(lib, kw, status):
    assert call_norm(lib, **kw) == status, b.aq_last_error()
    assert b.aq_last_error().startswith("aq_qk_norm_rope:")


def call_backward(lib, qn=norm(), kn=norm(), rope=ROPE, pos=0x3000, T=5, dim=64, dqo=heads(A), q=heads(B), dq=heads(C), dqw=0x4000, dko=heads(D_),
                  k=heads(E), dk=heads(F), dkw=0x5000, ws=0x70000000, nbytes=1 << 24):
    return lib.aq_qk_norm_rope_backward(ref(qn), ref(kn), ref(rope), pos, T, dim, ref(dqo), ref(q), ref(dq), dqw, ref(dko), ref(k), ref(dk), dkw, ws,
                                        nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), b.AQ_ERR_SHAPE), (dict(dim=8), b.AQ_ERR_SHAPE), (dict(qn=None), b.AQ_ERR_INVALID_ARG), (dict(dqo=None), b.AQ_ERR_INVALID_ARG),
    (dict(q=None), b.AQ_ERR_INVALID_ARG), (dict(dq=None), b.AQ_ERR_INVALID_ARG), (dict(kn=None), b.AQ_ERR_INVALID_ARG),
    (dict(dko=None), b.AQ_ERR_INVALID_ARG), (dict(dk=None), b.AQ_ERR_INVALID_ARG), (dict(kn=None, dko=None, k=None, dk=None), b.AQ_ERR_INVALID_ARG),
    (dict(qn=norm(weight=0)), b.AQ_ERR_INVALID_ARG), (dict(qn=norm(eps=-1.0)), b.AQ_ERR_INVALID_ARG), (dict(pos=None), b.AQ_ERR_INVALID_ARG),
    (dict(dq=heads(C, n=3)), b.AQ_ERR_SHAPE), (dict(dq=heads(C, tok=64)), b.AQ_ERR_SHAPE), (dict(q=heads(B + 2)), b.AQ_ERR_ALIGNMENT),
    (dict(dqw=0x4002), b.AQ_ERR_ALIGNMENT), (dict(ws=0), b.AQ_ERR_INVALID_ARG), (dict(ws=0x70000008), b.AQ_ERR_ALIGNMENT),
    (dict(nbytes=100), b.AQ_ERR_WORKSPACE), (dict(dq=heads(B)), b.AQ_ERR_OVERLAP), (dict(dq=heads(A, tok=512)), b.AQ_ERR_OVERLAP),
    (dict(dk=heads(C + 64)), b.AQ_ERR_OVERLAP), (dict(dkw=0x4000), b.AQ_ERR_OVERLAP), (dict(dqw=0x1000), b.AQ_ERR_OVERLAP), (dict(ws=A), b.AQ_ERR_OVERLAP),
    (dict(dq=heads(D_)), b.AQ_ERR_OVERLAP), (dict(dk=heads(A)), b.AQ_ERR_OVERLAP),
])
def test_norm_backward_refusals(lib, kw, status):
    assert call_backward(lib, **kw) == status, b.aq_last_error()
    assert b.aq_last_error().startswith("aq_qk_norm_rope_backward:")


def test_norm_workspace(lib):
    size = lib.aq_qk_norm_rope_backward_workspace_bytes
    assert 0 < size(1, 64, 1, 0) <= size(100000, 256, 64, 8) < 1 << 20
    for bad in ((-1, 64, 1, 1), (1, 40, 1, 1), (1, 64, 0, 1), (1, 64, 1, -1)):
        assert size(*bad) == ctypes.c_size_t(-1).value


def test_cache_write_refusals(lib):
    cache = b.c_kv_cache(k=A, v=B, k_scale=0, v_scale=0, pages=4, page_size=16, kv_heads=2, head_dim=64, type=b.AQ_KV_BF16)

    def call(rope=None, pos=0, q=0, qh=0, o=0, qn=None, kn=None):
        return lib.aq_kv_write_norm(ref(cache), 0x2000, 3, C, 128, 64, C + 0x100000, 128, 64, ref(rope), pos, q, qh, 256, 64, o, 256, 64, ref(qn), ref(kn), None)

    assert call(qn=norm()) == b.AQ_ERR_INVALID_ARG                        # a norm of queries that are not there
    assert call(q=D_, qh=4, o=E, kn=norm()) == b.AQ_ERR_INVALID_ARG       # queries with nothing to do to them
    assert call(kn=norm(eps=0.0)) == b.AQ_ERR_INVALID_ARG
    assert call(kn=norm(weight=0x1002)) == b.AQ_ERR_ALIGNMENT
    assert call(kn=norm(weight=A + 16)) == b.AQ_ERR_OVERLAP
    assert call(q=D_, qh=4, o=E, qn=norm(weight=E + 32)) == b.AQ_ERR_OVERLAP


# ---- products with NVFP4 weights ----
def weight(q=A, ldq=72, sf=B, g=0x1000, layout=0, out=40, inp=144):
    return b.c_nvfp4_weight(q, ldq, sf, g, layout, out, inp)


def call_linear(lib, ws=None, n=None, x=C, M=3, ldx=144, ys=None, lds=None):
    ws = [weight()] if ws is None else ws
    k = max(1, len(ws))
    ys, lds = [D_ + (i << 20) for i in range(k)] if ys is None else ys, [40] * k if lds is None else lds
    return lib.aq_nvfp4_linear_multi((b.c_nvfp4_weight * k)(*ws), len(ws) if n is None else n, x, M, ldx, (ctypes.c_void_p * k)(*ys), (ctypes.c_int64 * k)(*lds), None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), b.AQ_ERR_INVALID_ARG), (dict(n=4), b.AQ_ERR_INVALID_ARG), (dict(M=-1), b.AQ_ERR_SHAPE), (dict(ws=[weight(inp=0)]), b.AQ_ERR_SHAPE),
    (dict(ws=[weight(inp=136)]), b.AQ_ERR_SHAPE), (dict(ws=[weight(inp=65552, ldq=65552)]), b.AQ_ERR_UNSUPPORTED), (dict(ws=[weight(q=0)]), b.AQ_ERR_INVALID_ARG),
    (dict(ws=[weight(sf=0)]), b.AQ_ERR_INVALID_ARG), (dict(ws=[weight(g=0)]), b.AQ_ERR_INVALID_ARG), (dict(ws=[weight(layout=2)]), b.AQ_ERR_INVALID_ARG),
    (dict(ws=[weight(), weight(layout=1)]), b.AQ_ERR_INVALID_ARG), (dict(ws=[weight(), weight(inp=160, ldq=80)]), b.AQ_ERR_SHAPE),
    (dict(ws=[weight(out=0)]), b.AQ_ERR_SHAPE), (dict(ws=[weight(ldq=64)]), b.AQ_ERR_SHAPE), (dict(ws=[weight(ldq=76)]), b.AQ_ERR_ALIGNMENT),
    (dict(ws=[weight(q=A + 4)]), b.AQ_ERR_ALIGNMENT), (dict(ws=[weight(sf=B + 8)]), b.AQ_ERR_ALIGNMENT), (dict(ws=[weight(g=0x1002)]), b.AQ_ERR_ALIGNMENT),
    (dict(x=0), b.AQ_ERR_INVALID_ARG), (dict(x=C + 8), b.AQ_ERR_ALIGNMENT), (dict(ldx=148), b.AQ_ERR_ALIGNMENT), (dict(ldx=136), b.AQ_ERR_SHAPE),
    (dict(ys=[0]), b.AQ_ERR_INVALID_ARG), (dict(ys=[D_ + 1]), b.AQ_ERR_ALIGNMENT), (dict(lds=[39]), b.AQ_ERR_SHAPE), (dict(ys=[C + 64]), b.AQ_ERR_OVERLAP),
    (dict(ys=[A]), b.AQ_ERR_OVERLAP), (dict(ys=[B + 2]), b.AQ_ERR_OVERLAP), (dict(ys=[0x1000]), b.AQ_ERR_OVERLAP),
    (dict(ws=[weight(), weight()], ys=[D_, D_ + 40]), b.AQ_ERR_OVERLAP), (dict(ws=[weight(), weight()], ys=[D_, D_ + 60], lds=[80, 80]), b.AQ_ERR_OVERLAP),
])
def test_linear_refusals(lib, kw, status):
    assert call_linear(lib, **kw) == status, b.aq_last_error()
    assert b.aq_last_error().startswith("aq_nvfp4_linear:")


# ---- token scores ----
def call_scores(lib, x=A, ld=100, rows=3, vocab=100, type=0, tokens=0x1000, scale=1.0, lp=0x2000, lse=0x3000, h=0x4000, top=4, tl=0x5000, tt=0x6000):
    return lib.aq_token_logprobs(x, ld, rows, vocab, type, tokens, scale, lp, lse, h, top, tl, tt, None)


LOGITS = [
    (dict(rows=-1), b.AQ_ERR_SHAPE), (dict(vocab=0), b.AQ_ERR_SHAPE), (dict(vocab=(1 << 30) + 1), b.AQ_ERR_SHAPE), (dict(type=2), b.AQ_ERR_INVALID_ARG),
    (dict(scale=0.0), b.AQ_ERR_INVALID_ARG), (dict(scale=-1.0), b.AQ_ERR_INVALID_ARG), (dict(scale=float("nan")), b.AQ_ERR_INVALID_ARG),
    (dict(scale=float("inf")), b.AQ_ERR_INVALID_ARG), (dict(scale=9e-31), b.AQ_ERR_INVALID_ARG), (dict(scale=1.1e30), b.AQ_ERR_INVALID_ARG), (dict(x=0), b.AQ_ERR_INVALID_ARG), (dict(ld=99), b.AQ_ERR_SHAPE), (dict(x=A + 2), b.AQ_ERR_ALIGNMENT),
    (dict(x=A + 1, type=1), b.AQ_ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,status", LOGITS + [
    (dict(top=-1), b.AQ_ERR_UNSUPPORTED), (dict(top=33), b.AQ_ERR_UNSUPPORTED), (dict(top=4, vocab=3), b.AQ_ERR_UNSUPPORTED),
    (dict(tokens=0), b.AQ_ERR_INVALID_ARG), (dict(tl=0), b.AQ_ERR_INVALID_ARG), (dict(tt=0), b.AQ_ERR_INVALID_ARG),
    (dict(lp=0, lse=0, h=0, top=0), b.AQ_ERR_INVALID_ARG), (dict(lse=0x3002), b.AQ_ERR_ALIGNMENT), (dict(lse=A + 40), b.AQ_ERR_OVERLAP),
    (dict(lse=0x2008), b.AQ_ERR_OVERLAP), (dict(tt=0x5008), b.AQ_ERR_OVERLAP), (dict(h=0x1004), b.AQ_ERR_OVERLAP),
])
def test_scores_refusals(lib, kw, status):
    assert call_scores(lib, **kw) == status, b.aq_last_error()
    assert b.aq_last_error().startswith("aq_token_logprobs:")


def call_scores_backward(lib, x=A, ld=100, rows=3, vocab=100, type=0, tokens=0x1000, scale=1.0, lse=0x2000, h=0x3000, gp=0x4000, gh=0x5000, gl=0x6000, d=B,
                         ldd=100):
    return lib.aq_token_logprobs_backward(x, ld, rows, vocab, type, tokens, scale, lse, h, gp, gh, gl, d, ldd, None)


@pytest.mark.parametrize("kw,status", LOGITS + [
    (dict(lse=0), b.AQ_ERR_INVALID_ARG), (dict(d=0), b.AQ_ERR_INVALID_ARG), (dict(tokens=0), b.AQ_ERR_INVALID_ARG), (dict(gp=0), b.AQ_ERR_INVALID_ARG),
    (dict(gp=0, gh=0, gl=0, tokens=0), b.AQ_ERR_INVALID_ARG), (dict(h=0), b.AQ_ERR_INVALID_ARG), (dict(ldd=99), b.AQ_ERR_SHAPE),
    (dict(d=B + 2), b.AQ_ERR_ALIGNMENT), (dict(gl=0x6001), b.AQ_ERR_ALIGNMENT), (dict(d=A + 400), b.AQ_ERR_OVERLAP), (dict(d=A, ldd=104), b.AQ_ERR_OVERLAP),
    (dict(gh=B + 8), b.AQ_ERR_OVERLAP),
])
def test_scores_backward_refusals(lib, kw, status):
    assert call_scores_backward(lib, **kw) == status, b.aq_last_error()
    assert b.aq_last_error().startswith("aq_token_logprobs_backward:")


def test_empty_calls_do_nothing(lib):
    assert call_norm(lib, T=0, q=heads(0), qo=heads(0), k=heads(0), ko=heads(0), pos=None) == b.AQ_OK
    assert call_linear(lib, M=0, x=0, ys=[0]) == b.AQ_OK
    assert call_scores(lib, rows=0, x=0, tokens=0) == b.AQ_OK
    assert call_scores_backward(lib, rows=0, x=0, lse=0, d=0) == b.AQ_OK


def test_host_tensors_and_shapes_are_refused(lib):
    """The compiled marshalling: types, shapes and places, before any device work."""
    torch = pytest.importorskip("torch")
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    n = aq.HeadNorm(bf(64))
    w = aq.Nvfp4Weight(torch.zeros(8, 16, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8), torch.zeros(1))
    with pytest.raises(ValueError, match="CUDA device"):
        aq.aq_qk_norm_rope(bf(3, 2, 64), bf(3, 1, 64), n, n)
    with pytest.raises(ValueError, match="CUDA device"):
        aq.aq_qk_norm_rope_backward(bf(3, 2, 64), None, bf(3, 2, 64), None, n, None)
    with pytest.raises(ValueError, match="CUDA device"):
        aq.aq_nvfp4_linear(w, bf(3, 32))
    with pytest.raises(ValueError, match="CUDA device"):
        aq.aq_token_logprobs(bf(3, 32), i32(3))
    with pytest.raises(ValueError, match="CUDA device"):
        aq.aq_token_logprobs_backward(bf(3, 32), i32(3), torch.zeros(3), None, torch.zeros(3))
    for call, error in [
        (lambda: aq.aq_qk_norm_rope(bf(3, 2, 64), bf(4, 1, 64), n, n), ValueError), (lambda: aq.aq_qk_norm_rope(bf(3, 2, 32), q_norm=n), ValueError),
        (lambda: aq.aq_qk_norm_rope(torch.zeros(3, 2, 64), q_norm=n), TypeError), (lambda: aq.aq_qk_norm_rope(bf(3, 2, 64), q_norm=n, q_out=bf(3, 1, 64)), ValueError),
        (lambda: aq.aq_qk_norm_rope_backward(bf(3, 2, 64), None, bf(3, 2, 64), bf(3, 2, 64), n, n), ValueError),
        (lambda: aq.aq_qk_norm_rope_backward(bf(3, 2, 64), None, bf(3, 2, 64), None, None, None), ValueError),
        (lambda: aq.aq_nvfp4_linear(w, bf(3, 48)), ValueError), (lambda: aq.aq_nvfp4_linear(w, torch.zeros(3, 32)), TypeError),
        (lambda: aq.aq_nvfp4_linear(w, bf(3, 32), y=bf(3, 9)), ValueError), (lambda: aq.aq_nvfp4_linear_multi([], bf(3, 32)), ValueError),
        (lambda: aq.aq_nvfp4_linear_multi([w] * 4, bf(3, 32)), ValueError), (lambda: aq.aq_nvfp4_linear_multi([w, w], bf(3, 32), ys=[bf(3, 8)]), ValueError),
        (lambda: aq.aq_nvfp4_linear(aq.Nvfp4Weight(w.q, torch.zeros(8, 3, dtype=torch.uint8), w.global_scale), bf(3, 32)), ValueError),
        (lambda: aq.aq_nvfp4_linear(aq.Nvfp4Weight(w.q, w.sf, torch.zeros(2)), bf(3, 32)), ValueError),
        (lambda: aq.aq_nvfp4_linear(aq.Nvfp4Weight(w.q, w.sf, w.global_scale, aq.AQ_SF_128X4), bf(3, 32)), ValueError),
        (lambda: aq.aq_token_logprobs(bf(3, 32), i32(4)), ValueError), (lambda: aq.aq_token_logprobs(bf(3, 32), torch.zeros(3, dtype=torch.int64)), TypeError),
        (lambda: aq.aq_token_logprobs(bf(3, 32), i32(3), top=33), ValueError), (lambda: aq.aq_token_logprobs(torch.zeros(3, 32, dtype=torch.float16)), TypeError),
        (lambda: aq.aq_token_logprobs_backward(bf(3, 32), i32(3), torch.zeros(2), None, torch.zeros(3)), ValueError),
        (lambda: aq.aq_token_logprobs_backward(bf(3, 32), i32(3), torch.zeros(3), None, torch.zeros(3), dlogits=torch.zeros(3, 32)), TypeError),
    ]:
        with pytest.raises(error):
            call()
