"""Tensors of more than 2^31 values: rows past the border equal the same rows alone, and the rows
before it stay theirs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0
    torch.cuda.empty_cache()


def rows(gen, n, D):
    """n rows of D values, the same 1000 over and over but for the first and the last ten."""
    base = torch.randn(1000, D, device="cuda", generator=gen).bfloat16()
    x = base.repeat(-(-n // 1000), 1)[:n].contiguous()
    x[-10:] = torch.randn(10, D, device="cuda", generator=gen)
    return x


def test_sandwich_past_32_bits(rm):
    D, S = 16384, 140000  # 2.3e9 values
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, u = rows(gen, S, D)[None], rows(gen, S, D)[None]
    w = (1 + 0.1 * torch.randn(D, device="cuda", generator=gen)).bfloat16()
    rp, r = (torch.empty(S, dtype=torch.float32, device="cuda") for _ in range(2))
    res, out = rm.sandwich_rmsnorm_modulate(x, u, w, None, w, None, None, post_rstd_out=rp,
                                            rstd_out=r)
    g = rm.sandwich_rmsnorm_modulate_backward(u, res, w, None, w, None, x, out, rp, r)
    for part in (slice(0, 10), slice(S - 10, S)):
        a, b = rm.sandwich_rmsnorm_modulate(x[:, part], u[:, part], w, None, w, None, None)
        assert torch.equal(a, res[:, part]) and torch.equal(b, out[:, part])
        h = rm.sandwich_rmsnorm_modulate_backward(u[:, part], res[:, part], w, None, w, None,
                                                  x[:, part], out[:, part], rp[part], r[part])
        assert torch.equal(h.residual, g.residual[:, part])
        assert torch.equal(h.update, g.update[:, part])
    # the column sums: those of two halves added (fp32 sums of 140000 terms in items of up to 256
    # rows: each within 400 * 2^-24 of the magnitudes; compared in the 2-norm)
    halves = [rm.sandwich_rmsnorm_modulate_backward(
        u[:, p], res[:, p], w, None, w, None, x[:, p], out[:, p], rp[p], r[p], need_x=False)
        for p in (slice(0, S // 2), slice(S // 2, S))]
    for name in ("post_weight", "weight"):
        a = getattr(g, name).double()
        b = sum(getattr(h, name).double() for h in halves)
        assert (a - b).norm() <= 2 * 400 * 2.0 ** -24 * S ** 0.5 * a.norm()


def test_quantize_and_product_past_32_bits(rm):
    K, M = 16384, 140000
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = rows(gen, M, K)
    q = rm.mxfp4_quantize(x)
    y = rm.mxfp4_dequantize(q)
    for part in (slice(0, 10), slice(M - 10, M)):
        p = rm.mxfp4_quantize(x[part].contiguous())
        assert torch.equal(p.packed, q.packed[part])
        assert torch.equal(rm.mxfp4_dequantize(p), y[part])
    del y, q
    # a result of as many values
    w = rm.mxfp4_quantize(torch.randn(16384, 64, device="cuda", generator=gen).bfloat16())
    z = x[:, :64].contiguous()
    res = x  # as residual, in place
    last = res[-200:].clone()
    out = rm.mxfp4_linear(z, w, residual=res, out=res)
    want = rm.mxfp4_linear(z[-200:].contiguous(), w, residual=last)
    assert torch.equal(out[-200:], want)
