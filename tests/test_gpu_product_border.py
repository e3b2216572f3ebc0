"""The 4-bit product around 128 rows, where another kernel takes over that sums K in another order: up to
128 rows the sum is joined from parts of K, past them it runs through.  A row's result has the same bits
among the calls on either side, and on both sides it is within the bound of its definition: every step of
64 values adds to a running sum with an error of at most 2^-23 of the magnitudes summed, up to seven
additions join the parts with 2^-24 each, and the stored value is rounded once."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


@pytest.mark.parametrize("N,K", [(4096, 4096), (264, 16384), (9856, 1056)])
def test_both_sides_of_128_rows(rm, N, K):
    gen = torch.Generator(device="cuda").manual_seed(N + K)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen).half()  # noqa: E731
    x, w = rm.mxfp4_quantize(n(300, K)), rm.mxfp4_quantize(n(N, K) * K ** -0.5)
    a, b = (rm.mxfp4_dequantize(q, dtype=torch.float16).double() for q in (x, w))
    want, size = a @ b.T, a.abs() @ b.abs().T
    bound = 2.0 ** -11 * want.abs() + (K / 64 * 2.0 ** -23 + 7 * 2.0 ** -24) * size + 2.0 ** -24
    rows = rm.mxfp4_dequantize(x, dtype=torch.float16)  # quantised again they are themselves

    def product(m):
        out = rm.mxfp4_linear(rows[:m].contiguous(), w)
        assert out.isfinite().all()
        assert ((out.double() - want[:m]).abs() <= bound[:m]).all(), m
        return out

    few = [product(m) for m in (1, 16, 127, 128)]
    many = [product(m) for m in (129, 130, 257, 300)]
    for side in (few, many):
        for out in side[:-1]:
            assert torch.equal(out, side[-1][:out.shape[0]])
