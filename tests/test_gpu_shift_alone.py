"""The gradient of a shift without a scale, on the GPU, against the definition in float64 and against
the same call with a scale of zeros.  Bounds as in test_gpu_sandwich: column sums of go alone, whose
terms are exact, so a sum of n of them is within n 2^-24 of the magnitudes summed."""
import pytest
import torch

import _sandwich as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,S,D,rows", [(1, 5, 72, 1), (3, 21, 1024, 3), (3, 21, 1024, 1),
                                        (2, 9, 8456, 2)])
def test_shift_alone(rm, B, S, D, rows, dtype):
    gen = torch.Generator(device="cuda").manual_seed(D + rows)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(dtype)  # noqa: E731
    x, u, go, gr = n(B, S, D), n(B, S, D), n(B, S, D), n(B, S, D)
    shift = n(rows, 1, 2 * D)[..., D:]
    rp, r = (torch.empty(B * S, device="cuda") for _ in range(2))
    res, out = rm.sandwich_rmsnorm_modulate(x, u, shift=shift, post_rstd_out=rp, rstd_out=r)
    want, size = ref.norm(res, None, None, shift, 1e-6)
    assert ((out.double() - want).abs() <=
            torch.finfo(dtype).eps / 2 * want.abs() + 64 * 2.0 ** -24 * size + 1e-7).all()
    g = rm.sandwich_rmsnorm_modulate_backward(u, res, None, None, None, None, gr, go, rp, r,
                                              shift=shift)
    assert g.scale is None and g.shift.shape == (rows, D)
    want = ref.columns(go.double(), rows)
    bound = B * S * 2.0 ** -24 * ref.columns(go.double().abs(), rows)
    assert ((g.shift.double() - want).abs() <= bound).all()
    zeros = torch.zeros(rows, 1, D, dtype=dtype, device="cuda")
    h = rm.sandwich_rmsnorm_modulate_backward(u, res, None, None, None, zeros, gr, go, rp, r)
    assert torch.equal(g.shift, h.shift) and torch.equal(g.residual, h.residual)
    assert torch.equal(g.update, h.update)
