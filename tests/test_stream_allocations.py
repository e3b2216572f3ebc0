"""Where the sandwich and 4-bit calls allocate what they return, without a GPU.  A tensor belongs to the
memory pool of the stream that is current when it is made: freed, its memory goes to the next
allocation there, ordered by that stream alone.  So a call on another stream has to make its results
(and its workspace) under that one, or something else could be given the memory that it still writes;
and the caller's stream, which reads the results, has to be known to the pool."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

B, S, D = 2, 4, 64
HERE, SAME, SIDE = (SimpleNamespace(cuda_stream=i, device=torch.device("cpu")) for i in (0, 0, 7))


@pytest.fixture
def rm(monkeypatch):
    from rmsnorm_modulate_gb300 import _build

    _build.build()
    import rmsnorm_modulate_gb300 as rm

    state = SimpleNamespace(now=None, made={}, shared={})

    @contextlib.contextmanager
    def stream(s):
        before, state.now = state.now, s
        yield
        state.now = before

    def made(make):
        def call(*args, **kw):
            t = make(*args, **kw)
            state.made[id(t)] = (t, state.now)
            return t
        return call

    def record(t, s):
        state.shared[id(t)] = s

    monkeypatch.setattr(rm, "_bf16", lambda t, name, dtype=torch.bfloat16: t)
    monkeypatch.setattr(rm, "_call_on", lambda device, stream, name, *args: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.now or HERE)
    monkeypatch.setattr(torch.Tensor, "record_stream", record)
    monkeypatch.setattr(torch, "empty", made(torch.empty))
    monkeypatch.setattr(torch, "empty_like", made(torch.empty_like))
    rm.state = state
    yield rm
    del rm.state


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def calls(rm):
    x, stat, row = zeros(B, S, D), torch.zeros(B * S), zeros(B, 1, D)
    w = rm.Mxfp4(zeros(16, D // 2, dtype=torch.uint8), zeros(512, dtype=torch.uint8))
    q = rm.Mxfp4(zeros(B, S, D // 2, dtype=torch.uint8), zeros(512, dtype=torch.uint8))
    return {
        "forward": lambda **k: rm.sandwich_rmsnorm_modulate(x, x, scale=row, shift=row, **k),
        "backward": lambda **k: rm.sandwich_rmsnorm_modulate_backward(
            x, x, row[0, 0], row, row[0, 0], row, x, x, stat, stat, **k),
        "rms": lambda **k: rm.rmsnorm_modulate_backward(x, row[0, 0], row, x, stat, **k),
        "quantize": lambda **k: rm.mxfp4_quantize(x, **k),
        "dequantize": lambda **k: (rm.mxfp4_dequantize(q, **k),),
        "linear": lambda **k: (rm.mxfp4_linear(x, w, **k),),
    }


@pytest.mark.parametrize("name", ["forward", "backward", "rms", "quantize", "dequantize", "linear"])
def test_results_belong_to_the_call_s_stream(rm, name):
    got = calls(rm)[name](stream=SIDE)
    assert len(got) >= 1
    for t in got:
        assert rm.state.made[id(t)][1] is SIDE
        assert rm.state.shared[id(t)] is HERE
    assert all(s is SIDE for _, s in rm.state.made.values())  # the workspace too


@pytest.mark.parametrize("name", ["forward", "backward", "rms", "quantize", "dequantize", "linear"])
def test_results_on_the_current_stream(rm, name):
    for t in (*calls(rm)[name](), *calls(rm)[name](stream=SAME)):
        assert rm.state.made[id(t)][1] is None and id(t) not in rm.state.shared


def test_given_results_stay_the_caller_s(rm):
    x, out = zeros(B, S, D), zeros(B, S, D)
    a, b = rm.sandwich_rmsnorm_modulate(x, x, res_out=x, out=out, stream=SIDE)
    assert a is x and b is out
    q = rm.Mxfp4(zeros(B, S, D // 2, dtype=torch.uint8), zeros(512, dtype=torch.uint8))
    assert rm.mxfp4_quantize(x, out=q, stream=SIDE) is q
    assert rm.mxfp4_dequantize(q, out=out, stream=SIDE) is out
    w = rm.Mxfp4(zeros(D, D // 2, dtype=torch.uint8), zeros(512, dtype=torch.uint8))
    assert rm.mxfp4_linear(q, w, out=out, stream=SIDE) is out
    assert not rm.state.made and not rm.state.shared
    # rows that are quantised on the way need memory of that stream
    assert rm.mxfp4_linear(x, w, out=out, stream=SIDE) is out
    assert [s for _, s in rm.state.made.values()] == [SIDE]


@pytest.mark.parametrize("name", ["forward", "backward", "rms", "quantize", "dequantize", "linear"])
def test_a_stream_of_another_device_is_refused(rm, name):
    with pytest.raises(ValueError):
        calls(rm)[name](stream=SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 1)))
    assert all(s is None for _, s in rm.state.made.values())
