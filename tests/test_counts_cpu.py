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
