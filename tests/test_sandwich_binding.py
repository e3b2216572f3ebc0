"""What the Python calls of the sandwich norms pass on, without a GPU: the library's entry replaced by
one that records its arguments, the checks that want a CUDA tensor by ones that do not."""
import pytest
import torch

B, S, D = 3, 4, 64


@pytest.fixture
def rm(monkeypatch):
    from rmsnorm_modulate_gb300 import _build

    _build.build()
    import rmsnorm_modulate_gb300 as rm

    calls = []
    monkeypatch.setattr(rm, "_bf16", lambda t, name, dtype=torch.bfloat16: t)
    monkeypatch.setattr(rm, "_call_on", lambda device, stream, name, *args: calls.append((name, args)))
    rm.calls = calls
    yield rm
    del rm.calls


# of sandwich_rmsnorm_modulate_backward's arguments
SCALE, MOD_STRIDE, GRAD_SCALE, GRAD_SHIFT = 6, 7, 22, 23


def backward(rm, scale, **kw):
    x = torch.zeros(B, S, D, dtype=torch.bfloat16)
    stat = torch.zeros(B * S)
    g = rm.sandwich_rmsnorm_modulate_backward(x, x, None, None, None, scale, x, x, stat, stat, **kw)
    return g, rm.calls[-1][1]


def rows(n, width=D):
    return torch.zeros(n, 1, width, dtype=torch.bfloat16)


@pytest.mark.parametrize("n", [1, B])
def test_shift_alone_gets_its_gradient(rm, n):
    shift = rows(n, 3 * D)[..., D:2 * D]  # a view into wider rows
    g, args = backward(rm, None, shift=shift)
    assert g.shift.shape == (n, D) and g.shift.dtype == torch.float32
    assert g.scale is None and args[SCALE] is None and args[GRAD_SCALE] is None
    assert args[GRAD_SHIFT] == g.shift.data_ptr()
    assert args[MOD_STRIDE] == (3 * D if n > 1 else 0)


def test_shift_beside_scale(rm):
    scale, shift = rows(B, 2 * D).chunk(2, -1)
    both, a = backward(rm, scale, shift=shift)
    one, b = backward(rm, scale)  # a gradient of shift comes with that of scale
    for g, args in ((both, a), (one, b)):
        assert g.scale.shape == g.shift.shape == (B, D) and args[MOD_STRIDE] == 2 * D
    with pytest.raises(ValueError):  # rows of another stride
        backward(rm, scale, shift=rows(B))
    with pytest.raises(ValueError):
        backward(rm, None, shift=rows(2))


def test_no_gradient_of_what_took_no_part(rm):
    assert backward(rm, None)[0].shift is None
    assert backward(rm, None, shift=rows(B), need_mod=False)[0].shift is None
    x = torch.zeros(B, S, D, dtype=torch.bfloat16)
    g = rm.sandwich_rmsnorm_modulate_backward(x, None, None, None, None, None, x, None,
                                              torch.zeros(B * S), None, shift=rows(B))
    assert g.shift is None and rm.calls[-1][1][GRAD_SHIFT] is None
