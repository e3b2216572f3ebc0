"""Where the 8-bit calls allocate what they return, without a GPU: a call on another stream makes its
results and its workspace under that one, and notes the caller's stream on them; what the caller gives
stays the caller's."""
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

    monkeypatch.setattr(rm, "_bf16", lambda t, name, dtype=torch.bfloat16: t)
    monkeypatch.setattr(rm, "_call_on", lambda device, stream, name, *args: None)
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: state.now or HERE)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: state.shared.__setitem__(id(t), s))
    monkeypatch.setattr(torch, "empty", made(torch.empty))
    monkeypatch.setattr(torch, "empty_like", made(torch.empty_like))
    rm.state = state
    yield rm
    del rm.state


def held(rm, *shape):
    rows = 1
    for n in shape[:-1]:
        rows *= n
    codes = torch.zeros(*shape, dtype=torch.uint8).view(torch.float8_e4m3fn)
    return rm.Mxfp8(codes, torch.zeros(rm.mxfp8_scale_bytes(rows, shape[-1]), dtype=torch.uint8))


def calls(rm):
    x, row, stat = (torch.zeros(B, S, D).bfloat16(), torch.zeros(B, 1, D).bfloat16(),
                    torch.zeros(B * S))
    q, w = held(rm, B, S, D), held(rm, 32, D)
    return {
        "norm": lambda **k: rm.add_rmsnorm_mxfp8(x, x, row[0, 0], row, row, keep=True, **k),
        "norm_backward": lambda **k: rm.rmsnorm_mxfp8_backward(q, row[0, 0], row, x, stat, **k),
        "quantize": lambda **k: rm.mxfp8_quantize(x, **k),
        "dequantize": lambda **k: (rm.mxfp8_dequantize(q, **k),),
        "transpose": lambda **k: rm.mxfp8_transpose(q, **k),
        "linear": lambda **k: (rm.mxfp8_linear(x, w, **k),),
        "linear8": lambda **k: rm.mxfp8_linear(q, w, quantize=True, keep=True, **k),
        "activation": lambda **k: rm.mxfp8_activation_backward(q, x, "silu", row, **k),
    }


NAMES = ["norm", "norm_backward", "quantize", "dequantize", "transpose", "linear", "linear8",
         "activation"]


def leaves(v):
    return [t for x in v for t in leaves(x)] if isinstance(v, tuple) else [v]


@pytest.mark.parametrize("name", NAMES)
def test_results_belong_to_the_call_s_stream(rm, name):
    got = leaves(calls(rm)[name](stream=SIDE))
    for t in got:
        assert rm.state.made[id(t)][1] is SIDE and rm.state.shared[id(t)] is HERE
    assert all(s is SIDE for _, s in rm.state.made.values())  # the workspace too


@pytest.mark.parametrize("name", NAMES)
def test_results_on_the_current_stream(rm, name):
    for t in leaves(calls(rm)[name]()) + leaves(calls(rm)[name](stream=SAME)):
        assert rm.state.made[id(t)][1] is None and id(t) not in rm.state.shared


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(rm, name):
    with pytest.raises(ValueError):
        calls(rm)[name](stream=SimpleNamespace(cuda_stream=7, device=torch.device("cuda", 1)))
    assert all(s is None for _, s in rm.state.made.values())


def test_given_results_stay_the_caller_s(rm):
    x, q, k, w = torch.zeros(B, S, D).bfloat16(), held(rm, B, S, D), held(rm, B, S, D), held(rm, 64, D)
    res, out, kept = rm.add_rmsnorm_mxfp8(x, x, res_out=x, out=q, keep=k, stream=SIDE)
    assert res is x and out is q and kept is k
    assert rm.mxfp8_quantize(x, out=q, stream=SIDE) is q
    assert rm.mxfp8_dequantize(q, out=x, stream=SIDE) is x
    t = held(rm, D, 32)
    assert rm.mxfp8_transpose(q, out=t, stream=SIDE) is t
    assert rm.mxfp8_linear(q, w, out=x, keep=k, stream=SIDE) == (x, k)
    assert not rm.state.made and not rm.state.shared
    # x itself, where there is nothing to add, is not the call's to note
    res, out, _ = rm.add_rmsnorm_mxfp8(x, stream=SIDE)
    assert res is x and id(x) not in rm.state.shared and id(out.codes) in rm.state.shared
