"""Sizes at the end of 32 bits: a call serves them or refuses them. The checks run on the host before any device work, so placeholder
pointers are never dereferenced."""
import ctypes

import pytest

from rank_weight_reconstruction_gb300 import binding as b, build_lib

MOST = 2 ** 31 - 1
FAR = 1 << 40      # apart from each other by more than any of these extents


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return b.load()


@pytest.mark.parametrize("outs", [(MOST,), (MOST - 14,), (1 << 30, 1 << 30), (MOST, MOST, MOST), (2 ** 31 - 32, 16, 1)])
@pytest.mark.parametrize("layout", [b.AQ_SF_LINEAR, b.AQ_SF_128X4])
def test_rows_of_weights_past_32_bits_are_refused(lib, outs, layout):
    """Tiles of 16 rows, 2^27 - 1 in a call at most: one more row than 2^31 - 16, in one weight or in all."""
    n = len(outs)
    ws = [b.c_nvfp4_weight((4 * i + 1) * FAR, 8, (4 * i + 2) * FAR, (4 * i + 3) * FAR, layout, o, 16) for i, o in enumerate(outs)]
    ys, lds = [(4 * i + 4) * FAR for i in range(n)], list(outs)
    st = lib.aq_nvfp4_linear_multi((b.c_nvfp4_weight * n)(*ws), n, 20 * FAR, 1, 16, (ctypes.c_void_p * n)(*ys), (ctypes.c_int64 * n)(*lds), None)
    assert st == b.AQ_ERR_SHAPE and "too many rows" in b.aq_last_error(), (st, b.aq_last_error())


def test_dimensions_past_32_bits_are_refused(lib):
    """Tensors with more rows or heads than the ABI's counts hold are not served in part."""
    torch = pytest.importorskip("torch")
    import rank_weight_reconstruction_gb300 as aq

    many = 1 << 31
    heads = lambda n: torch.zeros(16, dtype=torch.bfloat16).expand(1, n, 16)  # noqa: E731
    i32 = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(8, dtype=torch.uint8).expand(many, 8)
    norm, rope = aq.HeadNorm(torch.zeros(16, dtype=torch.bfloat16)), aq.Rope(torch.zeros(8, dtype=torch.int64))
    cache = aq.KvCache(*(torch.zeros(1, 1, 16, 16, dtype=torch.bfloat16) for _ in "kv"))
    y, one = torch.zeros(1, 1, 16, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int64)
    for call in (
        lambda: aq.aq_nvfp4_linear(aq.Nvfp4Weight(q, torch.zeros(1, dtype=torch.uint8), torch.ones(1)), torch.zeros(1, 16, dtype=torch.bfloat16)),
        lambda: aq.aq_rope(rope, i32, heads(many), y=heads(many)),
        lambda: aq.aq_qk_norm_rope(heads(many), q_norm=norm, q_out=heads(many)),
        lambda: aq.aq_qk_norm_rope(y, heads(many), norm, norm, q_out=y, k_out=heads(many)),
        lambda: aq.aq_qk_norm_rope_backward(heads(many), None, heads(many), None, norm, None, dq=heads(many)),
        lambda: aq.aq_kv_write(cache, y, y, one, rope=rope, pos=i32, q=heads(many), q_out=heads(many)),
        lambda: aq.aq_tree_attention(cache, heads(many), torch.tensor([0, 1], dtype=torch.int32), i32, i32[None], max_q=1, out=heads(many)),
    ):
        with pytest.raises(ValueError, match="2147483648 are more than 32 bits hold"):
            call()


@pytest.mark.parametrize("hq,hk", [((1 << 30) + 1, 0), (MOST, 0), (MOST, 1), (1 << 30, 1 << 30), (1, MOST)])
def test_heads_past_what_a_list_holds_are_refused(lib, hq, hk):
    """The heads of a token are walked as one list, counted in 32 bits: q's and k's, and in the cache's write the values' too."""
    rope, norm = b.c_rope(FAR, 16, 0, 1.0), b.c_head_norm(2 * FAR, 1e-6, 0.0)
    heads = lambda i, n: ctypes.byref(b.c_heads(i * FAR, 16 * n, 16, n)) if n else None  # noqa: E731
    p = ctypes.byref
    calls = {
        "aq_qk_norm_rope": lambda: lib.aq_qk_norm_rope(p(norm), p(norm) if hk else None, p(rope), 3 * FAR, 1, 16, heads(4, hq), heads(5, hq), heads(6, hk), heads(7, hk), None),
        "aq_qk_norm_rope_backward": lambda: lib.aq_qk_norm_rope_backward(
            p(norm), p(norm) if hk else None, p(rope), 3 * FAR, 1, 16, heads(4, hq), heads(5, hq), heads(6, hq), None, heads(7, hk), heads(8, hk), heads(9, hk), None, None, 0, None),
    }
    if not hk:
        calls["aq_rope"] = lambda: lib.aq_rope(p(rope), 3 * FAR, 1, hq, 16, 4 * FAR, 16, 16, 5 * FAR, 16, 16, 0, None)
    cache = b.c_kv_cache(k=10 * FAR, v=12 * FAR, k_scale=0, v_scale=0, pages=1, page_size=16, kv_heads=hk or 1, head_dim=16, type=b.AQ_KV_BF16)
    calls["aq_kv_write"] = lambda: lib.aq_kv_write(p(cache), 2 * FAR, 1, 14 * FAR, 16, 16, 16 * FAR, 16, 16, p(rope), 3 * FAR, 4 * FAR, hq, 16, 16, 5 * FAR, 16, 16, None)
    for who, call in calls.items():
        st, said = call(), b.aq_last_error()
        assert st == b.AQ_ERR_SHAPE and said.startswith(who + ":") and "more than 2^30" in said, (st, said)


def test_the_single_weight_entry_refuses(lib):
    """aq_nvfp4_linear of the C ABI checks as the call for several weights does."""
    def call(w, x=20 * FAR, M=3, ldx=16, y=21 * FAR, ldy=40):
        return lib.aq_nvfp4_linear(w, x, M, ldx, y, ldy, None)

    weight = lambda out=40, inp=16, g=3 * FAR: ctypes.byref(b.c_nvfp4_weight(FAR, 8, 2 * FAR, g, b.AQ_SF_LINEAR, out, inp))  # noqa: E731
    for st, want in ((call(None), b.AQ_ERR_INVALID_ARG), (call(weight(g=0)), b.AQ_ERR_INVALID_ARG), (call(weight(out=0)), b.AQ_ERR_SHAPE),
                     (call(weight(inp=24)), b.AQ_ERR_SHAPE), (call(weight(), ldx=8), b.AQ_ERR_SHAPE), (call(weight(), ldx=18), b.AQ_ERR_ALIGNMENT),
                     (call(weight(), x=0), b.AQ_ERR_INVALID_ARG), (call(weight(), y=0), b.AQ_ERR_INVALID_ARG), (call(weight(), ldy=39), b.AQ_ERR_SHAPE),
                     (call(weight(), y=20 * FAR + 64), b.AQ_ERR_OVERLAP), (call(weight(out=MOST), ldy=MOST, M=1), b.AQ_ERR_SHAPE), (call(weight(), M=0), b.AQ_OK)):
        assert st == want, (st, want, b.aq_last_error())
