"""Head norms, NVFP4 products and token scores on a stream that is not the current one: what they allocate stays theirs until their
kernels are through, and what they return until the current stream is. A stream is kept busy by a spin of bounded length; every
check is of values or of addresses handed out meanwhile."""
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq

pytestmark = pytest.mark.gpu

BUSY = 600_000_000     # clocks: about a third of a second


def inputs():
    g = torch.Generator(device="cuda").manual_seed(3)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, dq, dk = randn(64, 8, 128), randn(64, 2, 128), randn(64, 8, 128), randn(64, 2, 128)
    n = aq.HeadNorm(randn(128), offset=1.0)
    rope, pos = aq.rope_frequencies(128), torch.arange(64, dtype=torch.int32, device="cuda")
    byte = lambda *shape: torch.randint(0, 0x70, shape, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    w = [aq.Nvfp4Weight(byte(o, 128), byte(o, 16), torch.ones(1, device="cuda")) for o in (512, 100)]
    x, logits = randn(16, 256), randn(64, 5000)
    tok = torch.randint(0, 5000, (64,), generator=g, device="cuda", dtype=torch.int32)
    s = aq.aq_token_logprobs(logits, tok)
    return {
        "norm": lambda **kw: list(aq.aq_qk_norm_rope(q, k, n, n, rope, pos, **kw)),
        "norm_backward": lambda **kw: list(aq.aq_qk_norm_rope_backward(dq, dk, q, k, n, n, rope, pos, **kw)),
        "nvfp4": lambda **kw: aq.aq_nvfp4_linear_multi(w, x, **kw),
        "scores": lambda **kw: list(aq.aq_token_logprobs(logits, tok, top=9, **kw)),
        "scores_backward": lambda **kw: [aq.aq_token_logprobs_backward(logits, tok, s.lse, s.entropy, s.logprob, **kw)],
    }


CALLS = pytest.mark.parametrize("call", ["norm", "norm_backward", "nvfp4", "scores", "scores_backward"])


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
def test_a_call_behind_one_that_writes_its_inputs(call):
    """Calls one after another on one stream, inputs written just before: nothing is read too early."""
    run = inputs()[call]
    want = run()
    torch.cuda.synchronize()
    for _ in range(20):
        got = run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
