"""Calls on a stream that is not the current one: whose memory their results take, and what they hold.
Addresses are compared, so nothing here depends on how fast the streams run."""
import pytest
import torch

pytestmark = pytest.mark.gpu

B, S, D = 2, 96, 1024


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


@pytest.fixture(scope="module")
def calls(rm):
    gen = torch.Generator(device="cuda").manual_seed(3)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    x, u, go, gr, v = n(B, S, D), n(B, S, D), n(B, S, D), n(B, S, D), n(D)
    gate, scale, shift = n(B, 1, 3 * D).chunk(3, -1)
    w, q = rm.mxfp4_quantize(n(256, D)), rm.mxfp4_quantize(x)
    stat = torch.ones(B * S, device="cuda")
    torch.cuda.synchronize()
    return {
        "forward": lambda **k: rm.sandwich_rmsnorm_modulate(x, u, v, gate, v, scale, shift, **k),
        "backward": lambda **k: rm.sandwich_rmsnorm_modulate_backward(
            u, x, v, gate, v, scale, gr, go, stat, stat, **k),
        "rms": lambda **k: rm.rmsnorm_modulate_backward(x, v, scale, go, stat, gr, **k),
        "quantize": lambda **k: rm.mxfp4_quantize(x, **k),
        "dequantize": lambda **k: (rm.mxfp4_dequantize(q, **k),),
        "linear": lambda **k: (rm.mxfp4_linear(x, w, **k),),
    }


NAMES = ["forward", "backward", "rms", "quantize", "dequantize", "linear"]


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def apart(a, b):
    return all(x1 <= y0 or y1 <= x0 for x0, x1 in a for y0, y1 in b)


def like(shapes):
    return [torch.empty(s, dtype=t, device="cuda") for s, t in shapes]


@pytest.mark.parametrize("name", NAMES)
def test_results_of_a_side_stream(rm, calls, name):
    call, side = calls[name], torch.cuda.Stream()
    want = [t.clone() for t in call()]
    shapes = [(t.shape, t.dtype) for t in want]
    torch.cuda.synchronize()
    # memory that the current stream has just let go of is not given to the call
    before = like(shapes)
    taken = spans(before)
    del before
    got = call(stream=side)
    assert apart(spans(got), taken)
    # the current stream is not given the results' memory while the call may still write it
    taken = spans(got)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    del got
    got = call(stream=side)
    taken = spans(got)
    del got
    assert apart(spans(like(shapes)), taken)
    torch.cuda.synchronize()
    # nor the next call on that stream the memory of results that the current stream still reads
    got = call(stream=side)
    taken = spans(got)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(20_000_000)  # about 10 ms
    kept = [t.clone() for t in got]
    del got
    assert apart(spans(call(stream=side)), taken)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


@pytest.mark.parametrize("name", NAMES)
def test_side_stream_in_a_graph(rm, calls, name):
    call, side = calls[name], torch.cuda.Stream()
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = call(stream=side)
        here.wait_stream(side)
        kept = [t + 0 for t in got]
    for _ in range(3):
        for t in kept:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, want))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
