"""The 8-bit operators on no tokens: results of that shape, sums of zero."""
import pytest
import torch

pytestmark = pytest.mark.gpu

N = 64


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


@pytest.mark.parametrize("shape", [(0, N), (2, 0, N), (0, 3, N)])
@pytest.mark.parametrize("per_batch", [False, True])
def test_no_rows(rm, shape, per_batch):
    e = lambda: torch.empty(*shape, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    batches = shape[0] if len(shape) == 3 else 1
    row = torch.ones((batches, 1, N) if per_batch else (N,), device="cuda").bfloat16()
    w = rm.mxfp8_quantize(torch.ones(N, N, device="cuda").bfloat16())
    res, h, kept = rm.add_rmsnorm_mxfp8(e(), e(), None, row, row, keep=True)
    y, z = rm.mxfp8_linear(h, w, activation="silu", gate=row, residual=res, keep=True)
    assert res.shape == h.codes.shape == kept.codes.shape == y.shape == z.codes.shape == shape
    dz, grad_bias, grad_gate = rm.mxfp8_activation_backward(z, e(), "silu", row)
    rows = batches if per_batch and batches > 1 else 1
    assert dz.codes.shape == shape and torch.equal(grad_bias, torch.zeros(N, device="cuda"))
    assert torch.equal(grad_gate, torch.zeros(rows, N, device="cuda"))
    grads = rm.rmsnorm_mxfp8_backward(kept, torch.ones(N, device="cuda").bfloat16(), row, e(),
                                      torch.empty(0, device="cuda"))
    assert grads[0].shape == shape and torch.equal(grads[1], torch.zeros(N, device="cuda"))
    for g in grads[2:]:
        assert torch.equal(g, torch.zeros(rows, N, device="cuda"))
    with pytest.raises(ValueError):
        rm.mxfp8_transpose(dz)
