"""8-bit matrices of more than 2^31 values: rows past the border equal the same rows alone, and the
rows before it stay theirs."""
import pytest
import torch

pytestmark = pytest.mark.gpu

M, K = 140000, 16384  # 2.3e9 values
ENDS = (slice(0, 10), slice(M - 10, M))


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0
    torch.cuda.empty_cache()


def rows(seed):
    """M rows of K values, the same 1000 over and over but for the last ten."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    base = torch.randn(1000, K, device="cuda", generator=gen).bfloat16()
    x = base.repeat(M // 1000, 1)
    x[-10:] = torch.randn(10, K, device="cuda", generator=gen)
    return x


def same(rm, part, q):
    """part, a matrix of ten rows, and the values of the whole one q at the same rows."""
    return torch.equal(rm.mxfp8_dequantize(part), q)


def test_rows_and_transpose_past_32_bits(rm):
    x = rows(0)
    q = rm.mxfp8_quantize(x)
    y = rm.mxfp8_dequantize(q)
    for part in ENDS:
        assert same(rm, rm.mxfp8_quantize(x[part].contiguous()), y[part])
    del y
    t = rm.mxfp8_transpose(q)
    back = rm.mxfp8_dequantize(t)
    assert back.shape == (K, M)
    for part in (slice(0, 32), slice(M - 32, M)):
        want = rm.mxfp8_transpose(rm.mxfp8_quantize(x[part].contiguous()))
        assert same(rm, want, back[:, part])
    del back
    # and with the many along the rows: [K, M] turned once more
    values = rm.mxfp8_dequantize(rm.mxfp8_transpose(t))
    first = rm.mxfp8_dequantize(t)[-32:].contiguous()
    assert same(rm, rm.mxfp8_transpose(rm.mxfp8_quantize(first)), values[:, -32:])


def test_norm_past_32_bits(rm):
    x, u = rows(1)[None], rows(2)[None]
    gen = torch.Generator(device="cuda").manual_seed(3)
    w = (1 + 0.1 * torch.randn(K, device="cuda", generator=gen)).bfloat16()
    rstd = torch.empty(M, dtype=torch.float32, device="cuda")
    res, out, kept = rm.add_rmsnorm_mxfp8(x, u, w, keep=True, rstd_out=rstd)
    gx, gw, _, _ = rm.rmsnorm_mxfp8_backward(kept, w, None, x, rstd, grad_res=u)
    out, values = rm.mxfp8_dequantize(out)[0], rm.mxfp8_dequantize(kept)[0]
    for part in ENDS:
        a, b, c = rm.add_rmsnorm_mxfp8(x[:, part], u[:, part], w, keep=True)
        assert torch.equal(a, res[:, part])
        assert same(rm, b, out[None, part]) and same(rm, c, values[None, part])
        h = rm.rmsnorm_mxfp8_backward(c, w, None, x[:, part], rstd[part], grad_res=u[:, part])
        assert torch.equal(h[0], gx[:, part])
    # the column sum: of two halves added, each in fp32 sums of up to 400 terms in a row (2-norm)
    both = 0
    for part in (slice(0, M // 2), slice(M // 2, M)):
        c = rm.mxfp8_quantize(res[:, part])
        both = both + rm.rmsnorm_mxfp8_backward(c, w, None, x[:, part], rstd[part],
                                                need_x=False)[1].double()
    assert (gw.double() - both).norm() <= 2 * 400 * 2.0 ** -24 * M ** 0.5 * gw.double().norm()


@pytest.mark.parametrize("act,gated", [("gelu_tanh", False), ("silu", True)])
def test_activation_gradient_past_32_bits(rm, act, gated):
    x, g = rows(4), rows(5)
    gate = g[:1].clone() if gated else None
    q = rm.mxfp8_quantize(x)
    grad_z, _, _ = rm.mxfp8_activation_backward(q, g, act, gate)
    values = rm.mxfp8_dequantize(grad_z)
    for part in ENDS:
        h = rm.mxfp8_activation_backward(rm.mxfp8_quantize(x[part].contiguous()), g[part], act, gate)
        assert same(rm, h[0], values[part])


def test_product_past_32_bits(rm):
    x = rows(6)
    gen = torch.Generator(device="cuda").manual_seed(7)
    w = rm.mxfp8_quantize(torch.randn(K, 64, device="cuda", generator=gen).bfloat16())
    z = x[:, :64].contiguous()
    last = x[-200:].clone()
    want = rm.mxfp8_linear(z[-200:].contiguous(), w, residual=last)
    out = rm.mxfp8_linear(z, w, residual=x, out=x)  # in place
    assert torch.equal(out[-200:], want)
    del out, x
    y, k = rm.mxfp8_linear(z, w, activation="silu", quantize=True, keep=True)
    a, b = rm.mxfp8_linear(z[-200:].contiguous(), w, activation="silu", quantize=True, keep=True)
    assert torch.equal(rm.mxfp8_dequantize(y)[-200:], rm.mxfp8_dequantize(a))
    assert torch.equal(rm.mxfp8_dequantize(k)[-200:], rm.mxfp8_dequantize(b))
    # and as an operand: 140000 rows of 16384 columns against a few
    n = rm.mxfp8_quantize(torch.randn(64, K, device="cuda", generator=gen).bfloat16())
    p = rm.mxfp8_linear(y, n)
    assert torch.equal(p[-200:], rm.mxfp8_linear(a, n))
