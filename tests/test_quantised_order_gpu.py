"""Calls right behind what writes their inputs, on one stream: every kernel here may begin before the one before it has ended, and none may
read activations, positions, words or statistics until then. Inputs alternate between two sets, so that a call that read early would
give the other set's outputs; every output is kept and compared with what a call of its own set gives after a wait."""
import numpy as np
import pytest
import torch

import rank_weight_reconstruction_gb300 as aq
from rank_weight_reconstruction_gb300 import synth
from helpers import dev_theta
import test_nvfp4_linear_gpu as products

pytestmark = pytest.mark.gpu

ROWS, WIDE, LAST, TURNS = 2048, 4096, 8, 24      # a buffer of 16 MB; the calls read its last rows, which its writer's last blocks write


def sources():
    g = torch.Generator(device="cuda").manual_seed(11)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    return g, randn, [randn(ROWS, WIDE) for _ in range(2)]


def writers():
    """Name -> what writes set i into the buffer: a kernel of torch's, and kernels of the library that let the next one begin early."""
    g, randn, src = sources()
    heads = lambda t: t.view(ROWS, 32, 128)  # noqa: E731
    rope, pos, n = aq.rope_frequencies(128), torch.arange(ROWS, dtype=torch.int32, device="cuda"), aq.HeadNorm(randn(128))
    byte = lambda *shape: torch.randint(0, 0x70, shape, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    w, x = aq.Nvfp4Weight(byte(WIDE, 256), byte(WIDE, 32), torch.full((1,), 1e-4, device="cuda")), [randn(32, 512) for _ in range(2)]
    return {
        "torch": lambda i, buf: torch.mul(src[i], 1.0, out=buf),
        "rope": lambda i, buf: aq.aq_rope(rope, pos, heads(src[i]), y=heads(buf)),
        "norm": lambda i, buf: aq.aq_qk_norm_rope(heads(src[i]), q_norm=n, rope=rope, pos=pos, q_out=heads(buf)),
        "product": lambda i, buf: aq.aq_nvfp4_linear(w, x[i], y=buf[-32:]),
        "gradient": lambda i, buf: aq.aq_qk_norm_rope_backward(heads(src[i]), None, heads(src[1 - i]), None, n, None, rope, pos, dq=heads(buf)),
        "scores' gradient": lambda i, buf: aq.aq_token_logprobs_backward(src[i], None, torch.zeros(ROWS, device="cuda"), dlse=torch.ones(ROWS, device="cuda"), dlogits=buf),
    }


def readers(buf):
    """Name -> a call on the buffer's last rows."""
    r = np.random.RandomState(5)
    g = torch.Generator(device="cuda").manual_seed(12)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    ws = [products.weight(r, o, WIDE)[0] for o in (300, 60)]
    last = buf[-LAST:]
    heads = last.view(LAST, 32, 128)
    n, rope, pos, other = aq.HeadNorm(randn(128), offset=1.0), aq.rope_frequencies(128), torch.arange(LAST, dtype=torch.int32, device="cuda"), randn(LAST, 32, 128)
    tok, one = torch.arange(LAST, dtype=torch.int32, device="cuda"), torch.ones(LAST, device="cuda")
    cache, slots = aq.KvCache.empty(2, 16, 16, 128, aq.AQ_KV_E4M3), torch.arange(LAST, device="cuda")

    def backward():
        s = aq.aq_token_logprobs(last, tok)
        return [aq.aq_token_logprobs_backward(last, tok, s.lse, s.entropy, one, dentropy=one)]

    def write():
        q = aq.aq_kv_write(cache, heads[:, 16:], heads[:, :16], slots, rope=rope, pos=pos, q=heads, q_norm=n, k_norm=n)
        return [q, *aq.aq_kv_read(cache, slots)]

    return {
        "nvfp4": lambda: aq.aq_nvfp4_linear_multi(ws, last),
        "norm": lambda: list(aq.aq_qk_norm_rope(heads[:, :24], heads[:, 24:], n, n, rope, pos)),
        "norm_backward x": lambda: [t for t in aq.aq_qk_norm_rope_backward(other, None, heads, None, n, None, rope, pos) if t is not None],
        "norm_backward dy": lambda: [t for t in aq.aq_qk_norm_rope_backward(heads, None, other, None, n, None, rope, pos) if t is not None],
        "kv_write": write,
        "scores": lambda: list(aq.aq_token_logprobs(last, tok, top=9)),
        "scores_backward": backward,
    }


def alternate(write, call):
    """Set 0 and set 1 in turn, as they come and captured in a graph: each output is its own set's."""
    want = []
    for i in range(2):
        write(i)
        torch.cuda.synchronize()
        want.append([t.clone() for t in call()])
        torch.cuda.synchronize()
    assert not all(torch.equal(a, b) for a, b in zip(*want))      # the sets tell each other apart

    def turns():
        got = []
        for i in range(TURNS):
            write(i % 2)
            got.append(call())
        return got

    got = turns()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = turns()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for outs in (got, replayed):
        for i, out in enumerate(outs):
            assert all(torch.equal(a, b) for a, b in zip(out, want[i % 2])), i


@pytest.mark.parametrize("reader", ["nvfp4", "norm", "norm_backward x", "norm_backward dy", "kv_write", "scores", "scores_backward"])
@pytest.mark.parametrize("writer", ["torch", "rope", "norm", "product", "gradient", "scores' gradient"])
def test_a_call_behind_the_kernel_that_writes_its_input(writer, reader):
    buf = torch.zeros(ROWS, WIDE, dtype=torch.bfloat16, device="cuda")
    write = writers()[writer]
    alternate(lambda i: write(i, buf), readers(buf)[reader])


def test_small_inputs_written_just_before():
    """Positions, slots, words, row statistics, norm weights and scales of products, by a kernel of torch's each."""
    g, randn, _ = sources()
    small = {
        "pos": [torch.arange(5, dtype=torch.int32, device="cuda") * (i + 1) + 7 for i in range(2)],
        "slots": [torch.tensor(v, device="cuda") for v in ([0, 1, 2, 3, 4], [9, 8, 7, 6, 5])],
        "tok": [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 1, 2, 3, 4], [90, 80, 70, 60, 50])],
        "lse": [torch.full((5,), 5.0 + i, device="cuda") for i in range(2)],
        "weight": [randn(64) for _ in range(2)],
        "g": [torch.full((1,), 0.5 + i, device="cuda") for i in range(2)],
    }
    now = {k: torch.zeros_like(v[0]) for k, v in small.items()}
    q, k, z, x, one = randn(5, 4, 64), randn(5, 2, 64), randn(5, 1000), randn(5, 256), torch.ones(5, device="cuda")
    rope, n = aq.rope_frequencies(64), aq.HeadNorm(now["weight"], offset=1.0)
    byte = lambda *shape: torch.randint(0, 0x70, shape, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    w = aq.Nvfp4Weight(byte(48, 128), byte(48, 16), now["g"])
    cache, every = aq.KvCache.empty(1, 16, 2, 64), torch.arange(16, device="cuda")

    def write(name):
        return lambda i: torch.add(small[name][i], 0, out=now[name])

    def cached():
        cache.k.zero_(), cache.v.zero_()
        write("slots")(cached.turn % 2)
        aq.aq_kv_write(cache, k, k, now["slots"], rope=rope, pos=now["pos"], k_norm=n)
        cached.turn += 1
        return list(aq.aq_kv_read(cache, every))

    write("pos")(0), write("weight")(0)
    cached.turn = 0
    alternate(write("pos"), lambda: list(aq.aq_qk_norm_rope(q, k, n, n, rope, now["pos"])))
    alternate(write("pos"), lambda: [t for t in aq.aq_qk_norm_rope_backward(q, k, q, k, n, n, rope, now["pos"])])
    alternate(write("weight"), lambda: list(aq.aq_qk_norm_rope(q, k, n, n, rope, now["pos"])))
    alternate(lambda i: None, cached)
    alternate(write("tok"), lambda: list(aq.aq_token_logprobs(z, now["tok"], top=2)))
    alternate(write("lse"), lambda: [aq.aq_token_logprobs_backward(z, now["tok"], now["lse"], dlogprob=one)])
    alternate(write("g"), lambda: [aq.aq_nvfp4_linear(w, x)])


@pytest.mark.parametrize("layout", [aq.AQ_SF_LINEAR, aq.AQ_SF_128X4])
def test_a_product_right_behind_the_precompute_of_its_weight(layout):
    """The precompute lets nothing begin before its end, so its codes and scales serve the very next call."""
    ths = [dev_theta(synth.make_theta(("order", i), 2048, 1152, 8)) for i in range(2)]
    q, sf, g = aq.aq_precompute_nvfp4(ths[0], sf_layout=layout)
    x = sources()[1](3, 1152)
    alternate(lambda i: aq.aq_precompute_nvfp4(ths[i], sf_layout=layout, global_scale=g, scale_given=False, q=q, sf=sf),
              lambda: [aq.aq_nvfp4_linear(aq.Nvfp4Weight(q, sf, g, layout), x)])


def test_a_product_on_a_stream_beside_a_replay():
    """A graph of two products replayed on new inputs while a call on another stream, ordered behind the inputs, reads the same x."""
    r = np.random.RandomState(7)
    (w1, v1), (w2, v2) = products.weight(r, 96, 128), products.weight(r, 128, 96)
    x = products.tokens(r, 5, 128)
    mid, y = torch.empty(5, 96, dtype=torch.bfloat16, device="cuda"), torch.empty(5, 128, dtype=torch.bfloat16, device="cuda")

    def both():
        aq.aq_nvfp4_linear(w1, x, y=mid)
        aq.aq_nvfp4_linear(w2, mid, y=y)

    both()
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(10):
        x.copy_(products.tokens(r, 5, 128))
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        other = aq.aq_nvfp4_linear(w1, x, stream=side)
        torch.cuda.synchronize()
        products.check(mid, x, v1)
        products.check(y, mid, v2)
        assert torch.equal(other, mid)
