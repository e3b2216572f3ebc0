"""Gates that are not finite (fp16 overflows to Inf) in the activation's gradient: only rows that there
are count.  A column under an Inf whose gradients have one sign sums to that Inf, whatever the number of
rows; the scale bytes behind the last row stay zero; the other columns keep their bits."""
import numpy as np
import pytest
import torch

import _mx8

pytestmark = pytest.mark.gpu

N = 160
INF = float("inf")


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


@pytest.mark.parametrize("act", _mx8.ACTIVATIONS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("per_batch", [False, True])
@pytest.mark.parametrize("B,S", [(1, 1), (1, 5), (1, 127), (1, 128), (1, 200), (3, 1), (3, 77), (2, 128),
                                 (2, 130)])
def test_gate_that_is_not_finite(rm, B, S, per_batch, dtype, act):
    rng = np.random.default_rng(B * S)
    # positive z and g: every product with the gate has the gate's sign, and none is zero
    z = rm.mxfp8_quantize(torch.from_numpy(rng.uniform(0.5, 4.0, (B, S, N))).to(dtype).cuda())
    g = torch.from_numpy(rng.uniform(0.5, 4.0, (B, S, N))).to(dtype).cuda()
    gate = torch.from_numpy(rng.uniform(0.5, 2.0, (B if per_batch else 1, 1, N))).to(dtype).cuda()
    fine = rm.mxfp8_activation_backward(z, g, act, gate)
    bad = gate.clone()
    bad[:, :, 1], bad[-1, :, 40], bad[0, :, 159] = INF, -INF, float("nan")
    grad_z, grad_bias, grad_gate = rm.mxfp8_activation_backward(z, g, act, bad)

    want = (g.double() * _mx8.activation(act, _mx8.decoded(z))[1] * bad.double()).view(-1, N)
    blocks = torch.isfinite(want).view(-1, N // 32, 32).all(-1).cpu().numpy()
    codes, scales, flat = _mx8.shown(grad_z)
    fine_codes, fine_scales, _ = _mx8.shown(fine[0])
    assert np.array_equal(_mx8.tiles(scales, N), flat)  # zeros behind the rows
    assert np.array_equal(scales, np.where(blocks, fine_scales, 255))
    keep = np.repeat(blocks, 32, axis=1)
    assert np.array_equal(codes[keep], fine_codes[keep])

    total = want.sum(0)
    assert total[1] == INF and total[40] == -INF and torch.isnan(total[159])
    off = ~torch.isfinite(total)
    assert off.sum() == 3 and torch.equal(grad_bias[~off], fine[1][~off])
    assert torch.equal(torch.nan_to_num(grad_bias[off].double(), nan=7.0),
                       torch.nan_to_num(total[off], nan=7.0))
    assert torch.equal(grad_gate, fine[2])  # the gate is not in its own gradient
