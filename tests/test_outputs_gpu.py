"""Outputs that the binding makes: those who watch allocations through a dispatch mode see them, those who ask for deterministic memory
get it, and otherwise they are ordinary tensors."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import rank_weight_reconstruction_gb300 as aq

pytestmark = pytest.mark.gpu


class Seen(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.shapes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func.name().startswith("aten::empty"):
            self.shapes.append(tuple(out.shape))
        return out


def calls():
    """Name -> (call, shapes of what it allocates)."""
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q, k, pos, rope = randn(5, 4, 64), randn(5, 2, 64), i32(0, 1, 2, 3, 4), aq.rope_frequencies(64)
    n = aq.HeadNorm(randn(64), offset=1.0)
    cache, slots = aq.KvCache.empty(2, 16, 2, 64), torch.arange(5, device="cuda")
    aq.aq_kv_write(cache, k, k, slots)
    byte = lambda *shape: torch.randint(0, 0x70, shape, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    w = aq.Nvfp4Weight(byte(48, 128), byte(48, 16), torch.ones(1, device="cuda"))
    x, z, tok = randn(5, 256), randn(5, 300), i32(1, 2, 3, 4, 5)
    p = torch.softmax(torch.randn(6, 40, generator=g, device="cuda"), -1)
    draft = (p, i32(1, 2, 3, 4, 5), i32(0, 5), torch.rand(5, generator=g, device="cuda"), torch.rand(1, 40, generator=g, device="cuda") + 0.1)
    s = aq.aq_token_logprobs(z, tok)
    heads, kv = (5, 4, 64), (5, 2, 64)
    return {
        "rope": (lambda: aq.aq_rope(rope, pos, q), [heads]),
        "kv_write": (lambda: aq.aq_kv_write(cache, k, k, slots, rope=rope, pos=pos, q=q), [heads]),
        "kv_read": (lambda: aq.aq_kv_read(cache, slots), [kv, kv]),
        "attention": (lambda: aq.aq_tree_attention(cache, q, i32(0, 5), i32(0), i32(0, 1)[None], max_q=5, return_lse=True), [heads, (5, 4)]),
        "verify": (lambda: aq.aq_verify_drafts(*draft), [(1,), (1, 5), (1,)]),
        "norm": (lambda: aq.aq_qk_norm_rope(q, k, n, n, rope, pos), [heads, kv]),
        "norm_backward": (lambda: aq.aq_qk_norm_rope_backward(q, k, q, k, n, n, rope, pos), [heads, kv, (64,), (64,)]),
        "nvfp4": (lambda: aq.aq_nvfp4_linear(w, x), [(5, 48)]),
        "scores": (lambda: aq.aq_token_logprobs(z, tok, top=3), [(5 * 9,)]),
        "scores_backward": (lambda: aq.aq_token_logprobs_backward(z, tok, s.lse, None, s.lse), [(5, 300)]),
    }


def tensors(out):
    return [t for t in (out if isinstance(out, (tuple, list)) else [out]) if t is not None]


NAMES = pytest.mark.parametrize("name", ["rope", "kv_write", "kv_read", "attention", "verify", "norm", "norm_backward", "nvfp4", "scores", "scores_backward"])


@NAMES
def test_a_dispatch_mode_sees_what_a_call_allocates(name):
    call, shapes = calls()[name]
    want = tensors(call())
    with Seen() as seen:
        got = tensors(call())
    for s in shapes:
        assert s in seen.shapes, (s, seen.shapes)
        seen.shapes.remove(s)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@NAMES
def test_with_deterministic_memory(name):
    """The same outputs where new memory is filled first."""
    call, _ = calls()[name]
    want = tensors(call())
    torch.use_deterministic_algorithms(True)
    try:
        got = tensors(call())
    finally:
        torch.use_deterministic_algorithms(False)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@NAMES
def test_outputs_are_ordinary_tensors(name):
    """Their type, device and strides, a history of their own from there on, and none before."""
    for t in tensors(calls()[name][0]()):
        assert t.is_cuda and t.is_contiguous() and t.grad_fn is None and not t.requires_grad
        if t.is_floating_point():
            leaf = t.detach().float().requires_grad_()
            (leaf * 2).sum().backward()
            assert (leaf.grad == 2).all()
