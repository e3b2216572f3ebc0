"""The 8-bit product's fp32 results with an activation, 8-bit results and checkpoints, on both sides of 128
rows, and the activations themselves over fp32's range.

Bounds, with u = 2^-24 and p = act(z) / z.  An activation is z p(z).  SiLU's p = 1 / (1 + 2^x): x has the
rounding of log2(e) (0.3 u) and its own (u), so ln 2^x is off by at most 1.3 u |ln p|; the exponential is
good to 2^-22 = 4 u, the sum to u, the reciprocal to 2^-23 = 2 u, the product with z to u: 8 u.  GELU's
tanh form: of the argument the linear part has the constants' 1.4 u, the fused sum's u and the product's
u, the cubic part z^2's u more, and the constant's: under 4 u |ln p| in all (an emulation of the steps
with exact instructions: 2.8 u |ln p|).  GELU: e^(-z^2 / 2) has 2.3 u |ln p| from z^2, constant and
product, 4 u from the instruction; the polynomial's 8 u, products 3 u.  So (16 + 4 |ln p|) u.  Where
p < 2^-125 the factors leave fp32's normal range: then up to |z| 2^-125 is lost.
The product and the epilogue: as in test_gpu_mxfp8.py; an activation's slope is under 1.2."""
import numpy as np
import pytest
import torch

import _mx8

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


def ln_share(act, z):
    """|ln(act(z) / z)| in 64 bits."""
    if act is None:
        return torch.zeros_like(z)
    if act == "gelu":
        return torch.special.log_ndtr(z).abs()
    c = 2 * (2 / np.pi) ** 0.5
    return torch.nn.functional.logsigmoid(z if act == "silu" else c * (z + 0.044715 * z ** 3)).abs()


def act_slack(act, z, y):
    if act is None:
        return torch.zeros_like(y)
    k = ln_share(act, z)
    return (16 + 4 * k) * U * y.abs() + torch.where(k > 125 * np.log(2), z.abs() * 2.0 ** -125, 0.0)


@pytest.mark.parametrize("act", _mx8.ACTIVATIONS)
@pytest.mark.parametrize("M", [1, 130])
def test_activation_over_the_range(rm, M, act):
    # rows of zeros: z is the bias itself, every step of the activation's error its own
    f = np.float32
    z = np.concatenate([np.linspace(-120, 30, 300000), np.linspace(-4, 4, 100000),
                        np.exp2(np.linspace(-149, 62, 20000)), -np.exp2(np.linspace(-149, 62, 20000)),
                        [0.0, -0.0, 19.74, -19.74, 19.8, -19.8, 3e38, -3e38]]).astype(f)
    z = np.concatenate([z, np.ones(-z.size % 8, f)])
    bias = torch.from_numpy(z).cuda()
    zeros = np.zeros((M, 32), np.uint8)
    x = _mx8.held(rm, zeros, zeros[:, :1])
    w = rm.mxfp8_quantize(torch.ones(z.size, 32, dtype=torch.bfloat16, device="cuda"))
    y = rm.mxfp8_linear(x, w, bias=bias, activation=act, dtype=torch.float32)
    assert y.dtype == torch.float32 and torch.equal(y, y[:1].expand(M, -1))
    z = bias.double()
    want = _mx8.activation(act, z.clamp(-1e100, 1e100))[0]
    want = torch.where(z.abs() > 1e6, z.clamp(min=0.0) if act else z, want)
    off = (y[0].double() - want).abs()
    # (fp32's own smallest step, once)
    bound = act_slack(act, z.clamp(-1e6, 1e6), want) + 2.0 ** -149
    assert (off <= bound).all(), (off / bound).max()


def test_activation_of_values_that_are_not_finite(rm):
    bias = torch.ones(32, device="cuda")
    bias[3], bias[9] = float("inf"), float("nan")
    zeros = np.zeros((2, 32), np.uint8)
    x = _mx8.held(rm, zeros, zeros[:, :1])
    w = rm.mxfp8_quantize(torch.ones(32, 32, dtype=torch.bfloat16, device="cuda"))
    for act in _mx8.ACTIVATIONS:
        y = rm.mxfp8_linear(x, w, bias=bias, activation=act, dtype=torch.float32)
        assert (y[:, 3] == float("inf")).all() and torch.isnan(y[:, 9]).all()
        assert torch.isfinite(y).sum() == 60


@pytest.mark.parametrize("act", _mx8.ACTIVATIONS)
@pytest.mark.parametrize("B,S,N,K,kw", [
    (1, 9, 160, 512, dict(bias=True)),
    (1, 9, 160, 512, dict(bias=True, quantize=True, keep=True)),
    (2, 60, 4096, 96, dict(keep=True, gate="batch", residual=True)),
    (1, 128, 96, 4160, dict(bias=True, keep=True)),
    (1, 129, 96, 4160, dict(bias=True, keep=True)),
    (2, 100, 288, 640, dict(bias=True, quantize=True)),
    (3, 90, 672, 352, dict(bias=True, quantize=True, keep=True, gate="batch", residual=True)),
    (1, 700, 4128, 256, dict(bias=True, gate="one", quantize=True, keep=True)),
    (1, 500, 1024, 128, dict(keep=True, residual=True, inplace=True)),
])
def test_product_activation_and_blocks(rm, B, S, N, K, kw, act):
    rng = np.random.default_rng(B * S + N + K)
    made = []
    for rows, lower in ((B * S, 0), (N, 18 if act else 0)):  # arguments where the activation bends
        codes, e = _mx8.random_codes(rng, rows, K)
        e = e - np.uint8(lower)
        made.append((_mx8.held(rm, codes, e), torch.from_numpy(_mx8.values(codes, e)).cuda()))
    (a, av), (b, bv) = made
    f32 = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().cuda()  # noqa: E731
    bias = f32(N) if kw.get("bias") else None
    gate = f32(B if kw["gate"] == "batch" else 1, 1, 3 * N).chunk(3, -1)[1] if kw.get("gate") else None
    residual = f32(B, S, N) * 8 if kw.get("residual") else None
    z = (av @ bv.T).view(B, S, N)
    slack = ((K / 32 + 2) * 2.0 ** -23 * (av.abs() @ bv.abs().T)).view(B, S, N)
    if bias is not None:
        z = z + bias.double()
        slack = slack + U * z.abs()
    z_slack = slack
    y = _mx8.activation(act, z)[0]
    if act:
        slack = 1.2 * slack + 1.01 * act_slack(act, z, y) + 1e-37  # (the argument is off by its slack)
    if gate is not None:
        y = y * gate.double()
        slack = slack * gate.double().abs() + U * y.abs()
    if residual is not None:
        y = y + residual.double()
        slack = slack + U * (y.abs() + slack)
    keep, quantize = kw.get("keep", False), kw.get("quantize", False)
    out = rm.mxfp8_linear(rm.Mxfp8(a.codes.view(B, S, K), a.scales), b, bias=bias, activation=act,
                          gate=gate, residual=residual, dtype=torch.float32,
                          out=residual if kw.get("inplace") else None, quantize=quantize, keep=keep)
    if keep:
        out, kept = out
        _mx8.check_held(kept, z, z_slack)
    if quantize:
        _mx8.check_held(out, y, slack)
    else:
        assert out.dtype == torch.float32 and out.shape == y.shape
        off = (out.double() - y).abs() / (_mx8.step_of(y, torch.float32) + slack)
        assert (off <= 1.0).all(), off.max()
