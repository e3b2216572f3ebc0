"""Results of the 8-bit product written into its 16-bit rows' own storage: at the rows' start or not, in 16
or in 8 bits, the checkpoint too, and alike for the few rows that the product quantises itself and for
those quantised before it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

N, K = 64, 128  # a result's row takes half of the bytes of a row of x


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


def taken(t, at, shape, dtype):
    """A view of that many of t's bytes from byte `at` on."""
    n = dtype.itemsize
    for s in shape:
        n *= s
    return t.view(-1).view(torch.uint8)[at:at + n].view(dtype).view(shape)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("M", [1, 5, 32, 33, 140])
def test_results_in_the_rows_own_place(rm, M, dtype):
    gen = torch.Generator(device="cuda").manual_seed(M)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(dtype)  # noqa: E731
    x, w = n(M, K), rm.mxfp8_quantize(n(N, K))
    want, kept = rm.mxfp8_linear(x, w, keep=True)
    want8 = rm.mxfp8_linear(x, w, quantize=True)
    scales = lambda: torch.empty_like(kept.scales)  # noqa: E731
    bits = lambda q: q.codes.view(torch.uint8)  # noqa: E731
    for at in (0, 16, M * N * 2, M * (K - N) * 2):  # the last two end with x
        y = x.clone()
        out = taken(y, at, (M, N), dtype)
        rm.mxfp8_linear(y, w, out=out)
        assert torch.equal(out, want), at
        y = x.clone()
        out = rm.Mxfp8(taken(y, at, (M, N), torch.float8_e4m3fn), scales())
        rm.mxfp8_linear(y, w, out=out, quantize=True)
        assert torch.equal(bits(out), bits(want8)) and torch.equal(out.scales, want8.scales)
        y = x.clone()
        keep = rm.Mxfp8(taken(y, at, (M, N), torch.float8_e4m3fn), scales())
        out, _ = rm.mxfp8_linear(y, w, keep=keep)
        assert torch.equal(out, want) and torch.equal(bits(keep), bits(kept))
        assert torch.equal(keep.scales, kept.scales)


@pytest.mark.parametrize("M", [32, 33])
def test_scales_in_the_rows_own_place(rm, M):
    x = torch.randn(M, K, device="cuda").bfloat16()
    w = rm.mxfp8_quantize(torch.randn(N, K, device="cuda").bfloat16())
    want = rm.mxfp8_linear(x, w, quantize=True)
    out = rm.Mxfp8(torch.empty_like(want.codes), taken(x, 32, want.scales.shape, torch.uint8))
    rm.mxfp8_linear(x, w, out=out, quantize=True)
    assert torch.equal(out.codes.view(torch.uint8), want.codes.view(torch.uint8))
    assert torch.equal(out.scales, want.scales)


@pytest.mark.parametrize("M", [32, 33])
def test_a_residual_that_is_partly_written_is_refused(rm, M):
    x = torch.randn(M + 1, N, device="cuda").bfloat16()
    w = rm.mxfp8_quantize(torch.randn(N, N, device="cuda").bfloat16())
    before = x.clone()
    with pytest.raises(rm.RmsmodError):
        rm.mxfp8_linear(x[:M], w, residual=x[:M], out=x[1:])
    assert torch.equal(x, before)
