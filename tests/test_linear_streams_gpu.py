"""The linears on a stream that is not the current one, without a workspace of the caller's: it is zeroed in the given stream's
order and stays the call's until its kernels are through."""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from rank_weight_reconstruction_gb300 import synth

from helpers import dev_theta

pytestmark = pytest.mark.gpu

BUSY = 600_000_000     # clocks: about a third of a second


def calls():
    make = lambda name, out, inp: dev_theta(synth.make_theta(("streams", name), out, inp, 16))  # noqa: E731
    q, k, v = make("q", 512, 768), make("k", 256, 768), make("v", 256, 768)
    gate, up, down = make("gate", 1024, 768), make("up", 1024, 768), make("down", 768, 1024)
    r = np.random.RandomState(1)
    x = {M: torch.from_numpy(r.standard_normal((M, 768)).astype(np.float32)).to(torch.bfloat16).cuda() for M in (4, 300)}
    return {
        "linear-4": lambda **kw: [aq.aq_linear(q, x[4], **kw)],
        "linear-300": lambda **kw: [aq.aq_linear(q, x[300], **kw)],
        "qkv": lambda **kw: list(aq.aq_linear_qkv([q, k, v], x[4], **kw)),
        "multi": lambda **kw: list(aq.aq_linear_multi([gate, up], x[4], **kw)),
        "mlp": lambda **kw: [aq.aq_mlp(gate, up, down, x[4], **kw)],
        "precompute": lambda **kw: [aq.aq_precompute(q, **kw)],
        "nvfp4": lambda **kw: list(aq.aq_precompute_nvfp4(q, **kw)),
    }


CALLS = pytest.mark.parametrize("call", ["linear-4", "linear-300", "qkv", "multi", "mlp", "precompute", "nvfp4"])


def fill():
    return [torch.empty(1 << k, dtype=torch.uint8, device="cuda").fill_(0x55) for k in range(9, 25) for _ in range(3)]


@CALLS
@pytest.mark.parametrize("busy", ["given", "current"])
def test_work_on_the_current_stream_around_a_call_elsewhere(call, busy):
    run = calls()[call]
    want = run()
    side, current = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    run(stream=side)
    fill()
    torch.cuda.synchronize()
    with torch.cuda.stream(side if busy == "given" else current):
        torch.cuda._sleep(BUSY)
    got = run(stream=side.cuda_stream)
    held = fill()
    assert not (side if busy == "given" else current).query() and held
    torch.cuda.synchronize()
    assert all(torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8)) for a, b in zip(got, want))
    assert aq.aq_device_status() == aq.AQ_OK
    assert torch.cuda.current_stream() == current
