"""Calls on a stream that is not the current one: what they allocate stays theirs until their kernels are through, and what they
return until the current stream is. A stream is kept busy by a spin of bounded length; every check is of values or of addresses
handed out meanwhile."""
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq

pytestmark = pytest.mark.gpu

BUSY = 600_000_000     # clocks: about a third of a second


def inputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = aq.KvCache.empty(200, 64, 2, 128, aq.AQ_KV_E4M3)
    n = 9000
    slots = torch.arange(n, device="cuda")
    aq.aq_kv_write(cache, randn(n, 2, 128), randn(n, 2, 128), slots)
    table = torch.arange(200, dtype=torch.int32, device="cuda")[None]
    q, one = randn(64, 8, 128), randn(64, 2, 128)
    rope, pos = aq.rope_frequencies(128), torch.arange(64, dtype=torch.int32, device="cuda")
    p = torch.softmax(torch.randn(5, 4096, generator=g, device="cuda"), -1)
    noise = torch.empty(1, 4096, device="cuda").exponential_(generator=g)
    cu, ctx, vcu, tok, u = i32([0, 64]), i32([8936]), i32([0, 4]), i32([5, 6, 7, 8]), torch.rand(4, generator=g, device="cuda")
    return {
        "rope": lambda **kw: [aq.aq_rope(rope, pos, q, **kw)],
        "kv_write": lambda **kw: [aq.aq_kv_write(cache, one, one, slots[:64] + 9100, rope=rope, pos=pos, q=q, **kw)],
        "kv_read": lambda **kw: list(aq.aq_kv_read(cache, slots[:64], **kw)),
        "attention": lambda **kw: list(aq.aq_tree_attention(cache, q, cu, ctx, table, max_q=64, return_lse=True, **kw)),
        "verify": lambda **kw: list(aq.aq_verify_drafts(p, tok, vcu, u, noise, **kw)),
    }


CALLS = pytest.mark.parametrize("call", ["rope", "kv_write", "kv_read", "attention", "verify"])


@CALLS
@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_work_on_the_current_stream_behind_a_call_elsewhere(call, raw):
    """The current stream allocates and writes at once, while the other stream has not begun the call."""
    run = inputs()[call]
    want = run()
    fill = lambda: [torch.empty(1 << k, dtype=torch.uint8, device="cuda").fill_(0x55) for k in range(9, 27) for _ in range(3)]  # noqa: E731
    side = torch.cuda.Stream()
    run(stream=side)
    fill()                                       # kernels loaded, memory at hand
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    got = run(stream=side.cuda_stream if raw else side)
    held = fill()
    assert not side.query()                      # the call was still to come
    torch.cuda.synchronize()
    assert len(held) and all(torch.equal(a, b) for a, b in zip(got, want))


@CALLS
def test_outputs_read_on_the_current_stream_stay_until_then(call):
    """An output let go while the current stream has yet to read it is not the next call's on the other stream."""
    run = inputs()[call]
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    side.wait_stream(current)
    want = run()
    out = run(stream=side)
    current.wait_stream(side)
    torch.cuda._sleep(BUSY)
    copies, places = [t.clone() for t in out], {t.data_ptr() for t in out}
    del out
    more = [run(stream=side) for _ in range(4)]
    assert not current.query()
    assert not places & {t.data_ptr() for ts in more for t in ts}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))


@CALLS
def test_the_current_streams_own_memory_is_left_alone(call):
    """A block that the current stream freed, with work on it still to come, is not written by a call elsewhere."""
    run = inputs()[call]
    want = run()
    sizes = [t.numel() * t.element_size() for t in want] + [1 << 25]
    torch.cuda.synchronize()
    held = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda._sleep(BUSY)
    copies, places = [t.clone() for t in held], {t.data_ptr() for t in held}
    del held
    out = run(stream=side)
    assert not places & {t.data_ptr() for t in out}
    torch.cuda.synchronize()
    assert all(bool((t == 7).all()) for t in copies) and all(torch.equal(a, b) for a, b in zip(out, want))


def test_default_stream_by_its_handles():
    run = inputs()["attention"]
    want = run()
    for handle in (0, 1, 2, torch.cuda.default_stream()):
        got = run(stream=handle)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0])
    with pytest.raises(ValueError):
        run(stream=3)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        run(stream=0)
        assert torch.cuda.current_stream() == side
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
