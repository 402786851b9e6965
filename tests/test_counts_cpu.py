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
