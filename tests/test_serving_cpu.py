"""Refusals of the serving entry points (argument checks run on the host before any device work, so
placeholder pointers are never dereferenced), and the frequency tables, which are host work."""
import ctypes

import numpy as np
import pytest

from oracle import serving
from rank_weight_reconstruction_gb300 import binding as b, build_lib

A, B, C, D_, E = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return b.load()


def rope(**kw):
    return b.c_rope(**{**dict(freq=0x1000, rotary_dim=64, layout=0, magnitude=1.0), **kw})


def cache(**kw):
    return b.c_kv_cache(**{**dict(k=A, v=B, k_scale=0x60000000, v_scale=0x70000000, pages=4, page_size=16, kv_heads=2,
                                  head_dim=64, type=b.AQ_KV_E4M3), **kw})


@pytest.mark.parametrize("rule,code", [("none", 0), ("linear", 1), ("ntk", 2), ("yarn", 3), ("wavelength", 4)])
def test_frequencies(lib, rule, code):
    n, out, mag = 32, (ctypes.c_uint64 * 32)(), ctypes.c_float()
    par = b.c_rope_scaling(8.0, 4096.0, 32.0, 1.0)
    assert lib.aq_rope_frequencies(64, 500000.0, code, ctypes.byref(par), ctypes.cast(out, ctypes.c_void_p), ctypes.byref(mag)) == 0
    want, m = serving.rope_angles(64, 500000.0, rule, 8.0, 4096.0)
    got = np.array([v / 2.0 ** 64 for v in out]) * 2 * np.pi
    assert np.allclose(got, want, rtol=1e-12) and np.isclose(mag.value, m, rtol=1e-6) and len(got) == n


@pytest.mark.parametrize("args,status", [
    ((63, 1e4, 0, None), b.AQ_ERR_SHAPE), ((0, 1e4, 0, None), b.AQ_ERR_SHAPE), ((258, 1e4, 0, None), b.AQ_ERR_SHAPE),
    ((64, 1.0, 0, None), b.AQ_ERR_INVALID_ARG), ((64, float("nan"), 0, None), b.AQ_ERR_INVALID_ARG),
    ((64, 1e4, 5, (8, 4096, 32, 1)), b.AQ_ERR_INVALID_ARG), ((64, 1e4, 1, None), b.AQ_ERR_INVALID_ARG),
    ((64, 1e4, 1, (0.5, 0, 0, 0)), b.AQ_ERR_INVALID_ARG), ((64, 1e4, 3, (8, 0, 32, 1)), b.AQ_ERR_INVALID_ARG),
    ((64, 1e4, 4, (8, 4096, 1, 1)), b.AQ_ERR_INVALID_ARG), ((2, 1e4, 2, (8, 0, 0, 0)), b.AQ_ERR_SHAPE),
])
def test_frequencies_refusals(lib, args, status):
    dim, base, code, par = args
    out, mag = (ctypes.c_uint64 * 256)(), ctypes.c_float()
    p = None if par is None else ctypes.byref(b.c_rope_scaling(*map(float, par)))
    assert lib.aq_rope_frequencies(dim, base, code, p, ctypes.cast(out, ctypes.c_void_p), ctypes.byref(mag)) == status
    assert b.aq_last_error()


def call_rope(lib, r=None, pos=0x2000, T=3, heads=2, dim=64, x=A, xt=128, xh=64, y=B, yt=128, yh=64):
    r = rope() if r is None else r
    return lib.aq_rope(ctypes.byref(r) if r else None, pos, T, heads, dim, x, xt, xh, y, yt, yh, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(r=rope(freq=0)), b.AQ_ERR_INVALID_ARG), (dict(r=rope(layout=2)), b.AQ_ERR_INVALID_ARG),
    (dict(r=rope(rotary_dim=24)), b.AQ_ERR_SHAPE), (dict(r=rope(rotary_dim=128)), b.AQ_ERR_SHAPE),
    (dict(r=rope(freq=0x1004)), b.AQ_ERR_ALIGNMENT), (dict(T=-1), b.AQ_ERR_SHAPE), (dict(heads=0), b.AQ_ERR_SHAPE),
    (dict(dim=72), b.AQ_ERR_SHAPE), (dict(dim=272), b.AQ_ERR_SHAPE), (dict(pos=0), b.AQ_ERR_INVALID_ARG),
    (dict(x=0), b.AQ_ERR_INVALID_ARG), (dict(y=0), b.AQ_ERR_INVALID_ARG), (dict(x=A + 8), b.AQ_ERR_ALIGNMENT),
    (dict(xt=132), b.AQ_ERR_ALIGNMENT), (dict(xh=32), b.AQ_ERR_SHAPE), (dict(yt=64), b.AQ_ERR_SHAPE),
    (dict(yt=0), b.AQ_ERR_SHAPE), (dict(y=A + 128), b.AQ_ERR_OVERLAP), (dict(y=A, yt=256), b.AQ_ERR_OVERLAP),
    (dict(pos=B + 64), b.AQ_ERR_OVERLAP),
])
def test_rope_refusals(lib, kw, status):
    assert call_rope(lib, **kw) == status, b.aq_last_error()
    assert b.aq_last_error().startswith("aq_rope")


def test_empty_calls_do_nothing(lib):
    assert call_rope(lib, T=0, pos=0, x=0, y=0) == b.AQ_OK
    assert call_write(lib, T=0, slots=0, k=0, v=0) == b.AQ_OK
    assert call_read(lib, T=0, slots=0) == b.AQ_OK
    assert call_attention(lib, dict(batch=0)) == b.AQ_OK
    assert call_attention(lib, dict(total_q=0)) == b.AQ_OK
    assert call_verify(lib, batch=0, cu=0, p=0) == b.AQ_OK


def call_write(lib, c=None, slots=0x2000, T=3, k=C, kt=128, kh=64, v=C + 0x100000, vt=128, vh=64, r=None, pos=0, q=0, qh=0,
               qt=256, qhd=64, o=0, ot=256, oh=64):
    c = cache() if c is None else c
    return lib.aq_kv_write(ctypes.byref(c), slots, T, k, kt, kh, v, vt, vh, ctypes.byref(r) if r else None, pos, q, qh, qt, qhd,
                           o, ot, oh, None)


def call_read(lib, c=None, slots=0x2000, T=3, k=C, kt=128, kh=64, v=C + 0x100000, vt=128, vh=64):
    c = cache() if c is None else c
    return lib.aq_kv_read(ctypes.byref(c), slots, T, k, kt, kh, v, vt, vh, None)


CACHE = [
    (dict(type=2), b.AQ_ERR_INVALID_ARG), (dict(k=0), b.AQ_ERR_INVALID_ARG), (dict(k_scale=0), b.AQ_ERR_INVALID_ARG),
    (dict(type=0), b.AQ_ERR_INVALID_ARG), (dict(pages=0), b.AQ_ERR_SHAPE), (dict(kv_heads=0), b.AQ_ERR_SHAPE),
    (dict(page_size=48), b.AQ_ERR_SHAPE), (dict(page_size=8), b.AQ_ERR_SHAPE), (dict(page_size=512), b.AQ_ERR_SHAPE),
    (dict(head_dim=72), b.AQ_ERR_SHAPE), (dict(head_dim=272), b.AQ_ERR_SHAPE), (dict(k=A + 8), b.AQ_ERR_ALIGNMENT),
    (dict(v_scale=0x70000004), b.AQ_ERR_ALIGNMENT), (dict(v=A + 1024), b.AQ_ERR_OVERLAP),
]


@pytest.mark.parametrize("kw,status", CACHE)
def test_cache_refusals(lib, kw, status):
    c = cache(**kw)
    assert call_write(lib, c) == status and b.aq_last_error().startswith("aq_kv_write")
    assert call_read(lib, c) == status and b.aq_last_error().startswith("aq_kv_read")
    assert call_attention(lib, c=c) == status and b.aq_last_error().startswith("aq_tree_attention")


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), b.AQ_ERR_SHAPE), (dict(slots=0), b.AQ_ERR_INVALID_ARG), (dict(k=0), b.AQ_ERR_INVALID_ARG),
    (dict(r=rope()), b.AQ_ERR_INVALID_ARG), (dict(q=D_, qh=4, o=E), b.AQ_ERR_INVALID_ARG),
    (dict(r=rope(), pos=0x3000, q=D_, qh=4), b.AQ_ERR_INVALID_ARG), (dict(r=rope(), pos=0x3000, q=D_, o=E), b.AQ_ERR_SHAPE),
    (dict(r=rope(rotary_dim=80), pos=0x3000), b.AQ_ERR_SHAPE), (dict(kt=100), b.AQ_ERR_ALIGNMENT),
    (dict(k=A), b.AQ_ERR_OVERLAP), (dict(v=0x60000000), b.AQ_ERR_OVERLAP),
    (dict(r=rope(), pos=0x3000, q=D_, qh=4, o=D_ + 512), b.AQ_ERR_OVERLAP),
    (dict(r=rope(), pos=0x3000, q=D_, qh=4, o=C), b.AQ_ERR_OVERLAP),
    (dict(r=rope(), pos=0x3000, q=D_, qh=4, o=E, ot=128), b.AQ_ERR_SHAPE),
])
def test_kv_write_refusals(lib, kw, status):
    assert call_write(lib, **kw) == status, b.aq_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), b.AQ_ERR_SHAPE), (dict(slots=0), b.AQ_ERR_INVALID_ARG), (dict(k=0, v=0), b.AQ_ERR_INVALID_ARG),
    (dict(k=A), b.AQ_ERR_OVERLAP), (dict(v=C + 64), b.AQ_ERR_OVERLAP), (dict(vt=64), b.AQ_ERR_SHAPE),
    (dict(v=C + 0x100004), b.AQ_ERR_ALIGNMENT),
])
def test_kv_read_refusals(lib, kw, status):
    assert call_read(lib, **kw) == status, b.aq_last_error()


def draft(**kw):
    return b.c_draft_batch(**{**dict(batch=2, max_q=4, total_q=8, cu_q=0x2000, ctx=0x3000, page_table=0x4000, pages_per_seq=2,
                                     ld_table=2, mask=0, ld_mask=0, depth=0, window=0), **kw})


def call_attention(lib, d=None, c=None, q=C, heads=4, qt=256, qh=64, o=D_, ot=256, oh=64, lse=0, ws=0x80000000, ws_bytes=1 << 30):
    c, d = cache() if c is None else c, draft(**(d or {}))
    return lib.aq_tree_attention(ctypes.byref(c), ctypes.byref(d), q, heads, qt, qh, 0.125, o, ot, oh, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(c=cache(head_dim=80)), b.AQ_ERR_UNSUPPORTED), (dict(heads=3), b.AQ_ERR_SHAPE), (dict(heads=0), b.AQ_ERR_SHAPE),
    (dict(d=dict(batch=-1)), b.AQ_ERR_SHAPE), (dict(d=dict(total_q=-1)), b.AQ_ERR_SHAPE), (dict(d=dict(max_q=-1)), b.AQ_ERR_SHAPE),
    (dict(d=dict(window=-1)), b.AQ_ERR_INVALID_ARG), (dict(d=dict(cu_q=0)), b.AQ_ERR_INVALID_ARG),
    (dict(d=dict(page_table=0)), b.AQ_ERR_INVALID_ARG), (dict(d=dict(ld_table=1)), b.AQ_ERR_SHAPE),
    (dict(d=dict(mask=0x5000, ld_mask=0)), b.AQ_ERR_SHAPE), (dict(d=dict(mask=0x5004, ld_mask=1)), b.AQ_ERR_ALIGNMENT),
    (dict(q=0), b.AQ_ERR_INVALID_ARG), (dict(o=0), b.AQ_ERR_INVALID_ARG), (dict(q=C + 8), b.AQ_ERR_ALIGNMENT),
    (dict(qt=252), b.AQ_ERR_ALIGNMENT), (dict(ot=128), b.AQ_ERR_SHAPE), (dict(o=C), b.AQ_ERR_OVERLAP), (dict(o=A), b.AQ_ERR_OVERLAP),
    (dict(lse=D_ + 16), b.AQ_ERR_OVERLAP), (dict(lse=2), b.AQ_ERR_ALIGNMENT), (dict(ws=0), b.AQ_ERR_WORKSPACE),
    (dict(ws=0x80000010), b.AQ_ERR_WORKSPACE), (dict(ws_bytes=4096), b.AQ_ERR_WORKSPACE), (dict(ws=A), b.AQ_ERR_OVERLAP),
    (dict(ws=D_), b.AQ_ERR_OVERLAP), (dict(d=dict(batch=1 << 23, max_q=64)), b.AQ_ERR_SHAPE),
])
def test_attention_refusals(lib, kw, status):
    assert call_attention(lib, **kw) == status, b.aq_last_error()


def call_verify(lib, batch=2, vocab=100, cu=0x1000, tok=0x2000, par=0, nodes=6, most=4, p=A, ld_p=100, q=0, ld_q=100, rows=8,
                kind=0, u=0x3000, noise=B, ld_n=100, n=C, path=C + 0x1000, ld_path=4, cap=4, token=C + 0x2000):
    return lib.aq_verify_drafts(batch, vocab, cu, tok, par, nodes, most, p, ld_p, q, ld_q, rows, kind, u, noise, ld_n, n, path,
                                ld_path, cap, token, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), b.AQ_ERR_SHAPE), (dict(vocab=0), b.AQ_ERR_SHAPE), (dict(most=1025), b.AQ_ERR_UNSUPPORTED),
    (dict(kind=2), b.AQ_ERR_INVALID_ARG), (dict(cu=0), b.AQ_ERR_INVALID_ARG), (dict(p=0), b.AQ_ERR_INVALID_ARG),
    (dict(tok=0), b.AQ_ERR_INVALID_ARG), (dict(u=0), b.AQ_ERR_INVALID_ARG), (dict(noise=0), b.AQ_ERR_INVALID_ARG),
    (dict(path=0), b.AQ_ERR_INVALID_ARG), (dict(rows=7), b.AQ_ERR_SHAPE), (dict(ld_p=99), b.AQ_ERR_SHAPE),
    (dict(q=D_, ld_q=99), b.AQ_ERR_SHAPE), (dict(ld_n=99), b.AQ_ERR_SHAPE), (dict(ld_path=3), b.AQ_ERR_SHAPE),
    (dict(p=A + 2), b.AQ_ERR_ALIGNMENT), (dict(token=C + 2), b.AQ_ERR_ALIGNMENT), (dict(n=B), b.AQ_ERR_OVERLAP),
    (dict(token=C), b.AQ_ERR_OVERLAP),
])
def test_verify_refusals(lib, kw, status):
    assert call_verify(lib, **kw) == status, b.aq_last_error()


def test_workspace_size_refuses_what_the_call_refuses(lib):
    c, d = cache(), draft()
    assert lib.aq_tree_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(d), 3) == ctypes.c_size_t(-1).value
    assert lib.aq_tree_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(d), 4) != ctypes.c_size_t(-1).value


def test_binding_checks_types_before_pointers():
    torch = pytest.importorskip("torch")
    x = torch.zeros(3, 2, 64, dtype=torch.float32)
    r = b.Rope(torch.zeros(32, dtype=torch.int64))
    with pytest.raises(TypeError):
        b.aq_rope(r, torch.zeros(3, dtype=torch.int32), x)
    with pytest.raises(TypeError):
        b.aq_rope(r, torch.zeros(3, dtype=torch.int64), x.bfloat16())
    with pytest.raises(ValueError):
        b.aq_rope(r, torch.zeros(4, dtype=torch.int32), x.bfloat16())
    kv = b.KvCache.empty(2, 16, 2, 64, b.AQ_KV_E4M3, device="cpu")
    with pytest.raises(ValueError):
        b.aq_kv_write(kv, x[:, :1].bfloat16(), x.bfloat16(), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        b.aq_kv_read(b.KvCache(kv.k[:, :1], kv.v, kv.k_scale, kv.v_scale), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        b.aq_kv_read(b.KvCache(kv.k, kv.v), torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError):
        b.aq_verify_drafts(torch.zeros(4, 8, dtype=torch.float64), torch.zeros(3, dtype=torch.int32),
                           torch.tensor([0, 3], dtype=torch.int32), torch.zeros(3), torch.ones(1, 8))
    with pytest.raises(ValueError):
        b.aq_tree_attention(kv, torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.tensor([0, 2], dtype=torch.int32),
                            torch.tensor([1, 2], dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32), max_q=2)
    with pytest.raises(b.AqError):   # well-formed tensors on the host: refused by the library, not read
        b.aq_tree_attention(kv, torch.zeros(2, 3, 64, dtype=torch.bfloat16), torch.tensor([0, 2], dtype=torch.int32),
                            torch.tensor([1], dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32), max_q=2)


def test_binding_passes_no_host_pointer_on():
    torch = pytest.importorskip("torch")
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    r = b.Rope(torch.zeros(32, dtype=torch.int64))
    pos, slots = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    kv = b.KvCache.empty(2, 16, 2, 64, b.AQ_KV_E4M3, device="cpu")
    cu, one = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([1], dtype=torch.int32)
    calls = [lambda p: b.aq_rope(r, p, x), lambda p: b.aq_kv_write(kv, x, x, slots, rope=r, pos=p),
             lambda p: b.aq_kv_read(kv, slots.to(p.device)),
             lambda p: b.aq_tree_attention(kv, x, cu, one, torch.zeros(1, 2, dtype=torch.int32), max_q=3, depth=p),
             lambda p: b.aq_verify_drafts(torch.zeros(4, 8), p, cu, torch.zeros(3), torch.ones(1, 8))]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA device"):
            call(pos)
        with pytest.raises(ValueError, match="other tensors on"):   # of two devices
            call(pos.to("meta"))


def test_a_call_within_a_call_leaves_the_outer_ones_checks_alone():
    """A Rope whose table is made on access, by other calls: the outer call's tensors are still checked among themselves."""
    torch = pytest.importorskip("torch")
    x, pos = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)

    class Lazy:
        layout, magnitude = b.AQ_ROPE_HALF, 1.0

        def __init__(self, device):
            self.device = device

        @property
        def freq(self):
            with pytest.raises(ValueError, match="other tensors on"):
                b.aq_rope(b.Rope(torch.zeros(32, dtype=torch.int64, device="meta")), pos, x)
            return torch.zeros(32, dtype=torch.int64, device=self.device)

    kv = b.KvCache.empty(2, 16, 2, 64, b.AQ_KV_E4M3, device="cpu")
    slots = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="Rope.freq: on meta, the call's other tensors on cpu"):
        b.aq_kv_write(kv, x, x, slots, rope=Lazy("meta"), pos=pos)
    with pytest.raises(ValueError, match="CUDA device"):
        b.aq_kv_write(kv, x, x, slots, rope=Lazy("cpu"), pos=pos)


@pytest.mark.parametrize("stream", [None, 0])
def test_tensors_on_a_device_that_is_not_current_are_refused(stream):
    """Tensors without memory stand for those of a device that is not current; the refusal comes before any device work."""
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("such tensors cannot be made beside a device")
    from torch._subclasses.fake_tensor import FakeTensorMode
    with FakeTensorMode():
        make = lambda dtype: lambda *shape: torch.empty(*shape, dtype=dtype, device="cuda:1")  # noqa: E731
        bf16, i32, i64, f32 = (make(d) for d in (torch.bfloat16, torch.int32, torch.int64, torch.float32))
        rope, cache = b.Rope(i64(64)), b.KvCache(bf16(4, 2, 16, 128), bf16(4, 2, 16, 128))
        x, pos, slots = bf16(3, 2, 128), i32(3), i64(3)
        p, cu, u, noise, table, one = f32(4, 50), i32(2), f32(3), f32(1, 50), i32(1, 4), i32(1)
    for call in (lambda: b.aq_rope(rope, pos, x, stream=stream), lambda: b.aq_kv_write(cache, x, x, slots, stream=stream),
                 lambda: b.aq_kv_read(cache, slots, stream=stream),
                 lambda: b.aq_tree_attention(cache, x, cu, one, table, max_q=3, stream=stream),
                 lambda: b.aq_verify_drafts(p, pos, cu, u, noise, stream=stream)):
        with pytest.raises(ValueError, match="are on cuda:1, which is not the current device"):
            call()
