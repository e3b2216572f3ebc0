"""The microscaled 8-bit operators against their definition in 64 bits.

Quantisation and the move to blocks along the other axis are exact (power-of-two scales, one rounding
to a code), so codes and scale bytes are compared for equality.  The product's bound per element: its
fp32 accumulation, every step of 32 values adding to the running sum with an error of at most 2^-23 (a
truncation) of the magnitudes summed, and the epilogue's operations with 2^-24 of theirs (2^-17 for an
activation, whose approximate instructions and argument's rounding are good to that); then the
output's half step, eps / 2 of the result, or that of the 8-bit block."""
import numpy as np
import pytest
import torch

import _mx8

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


def rows_of(rng, rows, K, dtype):
    """Values whose blocks have many magnitudes."""
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-6, 7, (rows, 1)))
    x *= np.exp2(np.repeat(rng.integers(-4, 5, (rows, K // 32)), 32, axis=1))
    return torch.from_numpy(x).to(dtype)


# ---------------------------------------------------------------------------------------------
# rows to blocks, back, and across
# ---------------------------------------------------------------------------------------------

def check_blocks(rm, x):
    rows, K = x.shape
    q = rm.mxfp8_quantize(x.cuda())
    y = rm.mxfp8_dequantize(q, dtype=x.dtype)
    codes, e = _mx8.quantize(x.double().numpy())
    got, _, flat = _mx8.shown(q)
    fine = np.repeat(e != 255, 32, axis=1)
    assert np.array_equal(flat, _mx8.tiles(e, K))  # the padding's zeros too
    assert np.array_equal(got[fine], codes[fine])
    want = torch.from_numpy(_mx8.values(got, e)).to(x.dtype)
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (127, 96), (128, 128), (129, 160), (33, 4128),
                                    (257, 1056), (640, 512)])
def test_quantize(rm, rows, K, dtype):
    check_blocks(rm, rows_of(np.random.default_rng(rows + K), rows, K, dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_edges(rm, dtype):
    f = torch.finfo(dtype)
    x = torch.zeros(13, 64, dtype=dtype)
    x[1, 0], x[1, 40] = f.max, -f.max
    x[2, 0] = f.smallest_normal
    x[3, 5] = f.smallest_normal * f.eps  # the smallest subnormal
    x[4, 0] = float("nan")
    x[5, 33] = float("inf")
    x[6, 0] = -float("inf")
    x[7, :32] = (torch.arange(32) + 0.5) * 2.0 ** -9  # ties of the small codes, under 448
    x[7, 31] = 448.0
    x[8] = -0.0
    x[9, 0], x[9, 1] = 448.0, 3.0
    x[10, 0], x[10, 1] = 448.0 * (1 + f.eps), 3.0  # one step past the border
    x[11, 0], x[11, 1] = 1.5, f.max
    x[12] = torch.arange(64) + 16.5  # ties
    check_blocks(rm, x)


def test_quantize_every_bf16(rm):
    # each finite pattern against a block that keeps the scale at 2^0, then alone
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    alone = torch.zeros(1 << 11, 32, dtype=torch.bfloat16)
    alone[:, 0] = bits[::32]
    check_blocks(rm, alone)
    small = bits[bits.abs() <= 448]
    x = torch.full((-(-small.numel() // 31), 32), 448.0, dtype=torch.bfloat16)
    flat = torch.zeros(x.shape[0] * 31, dtype=torch.bfloat16)
    flat[:small.numel()] = small
    x[:, 1:] = flat.view(-1, 31)
    check_blocks(rm, x)


def test_dequantize_every_code_and_scale(rm):
    codes = np.repeat(np.arange(256, dtype=np.uint8).reshape(8, 32), 256, axis=0)
    e = np.tile(np.arange(256, dtype=np.uint8), 8)[:, None]
    for dtype in TYPES:
        y = rm.mxfp8_dequantize(_mx8.held(rm, codes, e), dtype=dtype).cpu()
        want = torch.from_numpy(_mx8.values(codes, e)).float().to(dtype)  # exact in fp32 or Inf
        assert torch.equal(torch.nan_to_num(y, nan=7.0), torch.nan_to_num(want, nan=7.0))


def test_leading_shape_and_empty(rm):
    x = rows_of(np.random.default_rng(5), 6, 64, torch.bfloat16)
    a, b = rm.mxfp8_quantize(x.view(2, 3, 64).cuda()), rm.mxfp8_quantize(x.cuda())
    assert a.codes.shape == (2, 3, 64) and a.codes.dtype == torch.float8_e4m3fn
    assert torch.equal(a.codes.view(torch.uint8).view(6, 64), b.codes.view(torch.uint8))
    assert torch.equal(a.scales, b.scales) and rm.mxfp8_dequantize(a).shape == (2, 3, 64)
    t = rm.mxfp8_transpose(a)
    assert t.codes.shape == (64, 32)
    assert torch.equal(t.codes.view(torch.uint8), rm.mxfp8_transpose(b).codes.view(torch.uint8))
    q = rm.mxfp8_quantize(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert q.codes.shape == (0, 64) and q.scales.numel() == 0
    assert rm.mxfp8_dequantize(q).shape == (0, 64)


def check_across(rm, codes, e):
    t = rm.mxfp8_transpose(_mx8.held(rm, codes, e))
    want, we = _mx8.across(codes, e)
    assert t.codes.shape == want.shape
    got, ge, flat = _mx8.shown(t)
    assert np.array_equal(ge, we)
    assert np.array_equal(flat, _mx8.tiles(we, want.shape[1]))
    fine = np.repeat(we != 255, 32, axis=1)
    assert np.array_equal(got[fine], want[fine])
    return t


@pytest.mark.parametrize("rows,K", [(1, 32), (31, 64), (32, 160), (33, 96), (100, 128), (128, 416),
                                    (129, 32), (300, 1056), (1030, 288)])
def test_transpose(rm, rows, K):
    rng = np.random.default_rng(rows * K)
    check_across(rm, *_mx8.random_codes(rng, rows, K))
    # what quantising gives: every block uses its scale; and scales that are far apart
    check_across(rm, *_mx8.quantize(rows_of(rng, rows, K, torch.float32).double().numpy()))
    check_across(rm, *_mx8.random_codes(rng, rows, K, 0, 255))


def test_transpose_edges(rm):
    rng = np.random.default_rng(8)
    codes, e = _mx8.random_codes(rng, 96, 64)
    codes[:32, 3] = 0  # a block of zeros, beside scales that are large
    codes[:32, 4] = 128
    codes[5, 7] = 127  # NaN
    codes[40, 9] = 255
    e[70, 1] = 255
    codes[:, 20] = 0
    codes[3, 20] = 1  # the smallest code alone, under any scale
    e[3, 0] = 254
    codes[:, 21] = 126
    e[64:, 0] = 0
    check_across(rm, codes, e)
    zeros = np.zeros((64, 32), np.uint8)
    check_across(rm, zeros, zeros[:, :1])
    check_across(rm, zeros, zeros[:, :1] + 254)


def test_transpose_twice_keeps_values(rm):
    # values of one binade's range lose nothing, either way
    rng = np.random.default_rng(4)
    x = torch.from_numpy(rng.integers(-8, 9, (160, 224)) * 0.25).bfloat16().cuda()
    q = rm.mxfp8_quantize(x)
    t = rm.mxfp8_transpose(q)
    assert torch.equal(rm.mxfp8_dequantize(t), x.t())
    assert torch.equal(rm.mxfp8_dequantize(rm.mxfp8_transpose(t)), x)


def test_transpose_ignores_what_lies_behind_its_rows(rm):
    rng = np.random.default_rng(2)
    codes, e = _mx8.random_codes(rng, 37, 64)
    q = _mx8.held(rm, codes, e)
    g = q.scales.view(-1, 32, 4, 4)
    r = torch.arange(128, device="cuda").view(4, 32).T
    g[(r >= 37).expand(g.shape[0], 32, 4)] = 255
    t = rm.mxfp8_transpose(q)
    want, we = _mx8.across(codes, e)
    got, ge, _ = _mx8.shown(t)
    assert np.array_equal(got, want) and np.array_equal(ge, we)


# ---------------------------------------------------------------------------------------------
# the product
# ---------------------------------------------------------------------------------------------

def make(rm, rng, rows, K):
    codes, e = _mx8.random_codes(rng, rows, K)
    return _mx8.held(rm, codes, e), torch.from_numpy(_mx8.values(codes, e)).cuda()


def check_product(rm, rng, B, S, N, K, dtype, bias=False, act=None, gate=None, residual=False,
                  inplace=False, quantize=False, keep=False):
    a, av = make(rm, rng, B * S, K)
    b, bv = make(rm, rng, N, K)
    if act:  # arguments where the activation bends
        b = rm.Mxfp8(b.codes, torch.clamp(b.scales.int() - 18, min=0).to(torch.uint8))
        bv = bv * 2.0 ** -18
    half = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype).cuda()  # noqa: E731
    bt = half(N) if bias else None
    gt = None
    if gate:  # a view into rows of three, as an adaLN projection gives it
        gt = half(B if gate == "batch" else 1, 1, 3 * N).chunk(3, -1)[1]
    rt = half(B, S, N) * 8 if residual else None
    z = (av @ bv.T).view(B, S, N)
    slack = ((K / 32 + 2) * 2.0 ** -23 * (av.abs() @ bv.abs().T)).view(B, S, N)
    if bias:
        z = z + bt.double()
        slack = slack + 2.0 ** -24 * z.abs()
    z_slack = slack
    y, slope = _mx8.activation(act, z)
    if act:
        # the slope is at most 1.13 in magnitude; products near 0 have a relative error
        slack = 1.2 * slack + 2.0 ** -17 * y.abs() + 1e-30
    if gate:
        y, slack = y * gt.double(), slack * gt.double().abs() + 2.0 ** -24 * (y * gt.double()).abs()
    if residual:
        y = y + rt.double()
        slack = slack + 2.0 ** -24 * y.abs()
    q = rm.Mxfp8(a.codes.view(B, S, K), a.scales)
    out = rm.mxfp8_linear(q, b, bias=bt, activation=act, gate=gt, residual=rt, dtype=dtype,
                          out=rt if inplace else None, quantize=quantize, keep=keep)
    if keep:
        out, kept = out
        assert kept.codes.shape == (B, S, N)
        _mx8.check_held(kept, z, z_slack)
    if quantize:
        assert out.codes.shape == (B, S, N)
        _mx8.check_held(out, y, slack)
        return out
    assert out.shape == (B, S, N) and out.dtype == dtype
    over = y.abs() > float(torch.finfo(dtype).max)
    off = ((out.double() - y).abs() / (_mx8.step_of(y, dtype) * (1 + 2.0 ** -10) + slack))[~over]
    assert not off.numel() or off.max().item() <= 1.0, (B, S, N, K, off.max().item())
    return out


SHAPES = [(1, 8, 32), (1, 4096, 64), (5, 264, 96), (8, 1000, 4096), (16, 128, 2080), (127, 256, 128),
          (128, 256, 256), (129, 248, 288), (200, 520, 1056), (640, 1536, 512), (1000, 3080, 736),
          (33, 72, 16384)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [*TYPES, torch.float32])
def test_product(rm, M, N, K, dtype):
    check_product(rm, np.random.default_rng(M + N + K), 1, M, N, K, dtype)


EPILOGUES = [
    (1, 7, 264, 512, dict(bias=True)),
    (3, 50, 136, 320, dict(gate="batch", residual=True)),
    (2, 129, 512, 1024, dict(bias=True, gate="shared", residual=True)),
    (2, 1, 4096, 256, dict(bias=True, gate="batch", residual=True, inplace=True)),
    (4, 33, 40, 64, dict(gate="batch")),
    (1, 300, 280, 2048, dict(residual=True, inplace=True)),
]


@pytest.mark.parametrize("dtype", [*TYPES, torch.float32])
@pytest.mark.parametrize("B,S,N,K,kw", EPILOGUES)
def test_product_epilogue(rm, B, S, N, K, kw, dtype):
    check_product(rm, np.random.default_rng(B * S + N), B, S, N, K, dtype, **kw)


@pytest.mark.parametrize("act", _mx8.ACTIVATIONS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,S,N,K,kw", [
    (1, 9, 160, 512, dict(bias=True)),
    (1, 9, 160, 512, dict(bias=True, quantize=True, keep=True)),
    (2, 60, 4096, 96, dict(keep=True, gate="batch", residual=True)),
    (2, 100, 288, 640, dict(bias=True, quantize=True)),
    (3, 90, 672, 352, dict(bias=True, quantize=True, keep=True, gate="batch", residual=True)),
    (1, 700, 4128, 256, dict(bias=True, quantize=True, keep=True)),
    (1, 500, 1024, 128, dict(keep=True, residual=True, inplace=True)),
])
def test_product_activation_and_blocks(rm, B, S, N, K, kw, dtype, act):
    check_product(rm, np.random.default_rng(B * S + N), B, S, N, K, dtype, act=act, **kw)


def test_product_of_integers_is_exact(rm):
    # codes whose products and sums are small integers: no rounding anywhere
    rng = np.random.default_rng(3)
    for M, N, K in ((40, 72, 32), (130, 264, 160), (8, 512, 512)):
        e, q = {}, {}
        for name, rows in (("a", M), ("b", N)):
            v = rng.integers(-6, 7, (rows, K)) * (rng.random((rows, K)) < 0.3)
            codes = _mx8.nearest(v.astype(np.float64))
            g = np.full((rows, K // 32), 127, np.uint8)
            e[name] = _mx8.values(codes, g)
            assert np.array_equal(e[name], v)
            q[name] = _mx8.held(rm, codes, g)
        want = e["a"] @ e["b"].T
        assert np.abs(want).max() < 2048
        for dtype in (torch.float16, torch.float32):
            out = rm.mxfp8_linear(q["a"], q["b"], dtype=dtype)
            assert np.array_equal(out.double().cpu().numpy(), want)


def test_product_quantises_its_rows(rm):
    rng = np.random.default_rng(9)
    x = rows_of(rng, 77, 608, torch.bfloat16).cuda()
    w, _ = make(rm, rng, 264, 608)
    a = rm.mxfp8_linear(x, w)
    assert torch.equal(a, rm.mxfp8_linear(rm.mxfp8_quantize(x), w))
    # a row's result does not depend on the rows beside it
    assert torch.equal(a[5:9], rm.mxfp8_linear(x[5:9].contiguous(), w))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K,kw", [
    (1, 8, 32, {}), (1, 4096, 4096, {}), (7, 264, 96, {}), (16, 136, 2080, dict(activation="silu")),
    (17, 96, 352, dict(quantize=True, keep=True)), (32, 4096, 4128, dict(keep=True)),
    (32, 128, 20480, {}), (33, 128, 160, {}), (5, 16384, 160, dict(quantize=True)),
])
def test_product_quantises_few_rows_itself(rm, M, N, K, kw, dtype):
    # the same bits as with rows that were quantised before
    rng = np.random.default_rng(M * N + K)
    x = rows_of(rng, M, K, dtype)
    x[M // 2, K // 2] = 0.0
    if M > 2:
        x[2, :32] = 0.0  # a block of zeros
    x = x.cuda()
    w, _ = make(rm, rng, N, K)
    a = rm.mxfp8_linear(x, w, dtype=dtype, **kw)
    b = rm.mxfp8_linear(rm.mxfp8_quantize(x), w, dtype=dtype, **kw)
    flat = lambda v: [t for u in v for t in flat(u)] if isinstance(v, tuple) else [v]  # noqa: E731
    for p, q in zip(flat(a), flat(b)):
        assert torch.equal(p.view(torch.uint8), q.view(torch.uint8))


def test_rows_do_not_depend_on_how_many_there_are(rm):
    # past 128 rows: narrow and wide tiles give a row the same bits
    rng = np.random.default_rng(10)
    x = rows_of(rng, 6000, 736, torch.bfloat16).cuda()
    w, _ = make(rm, rng, 2080, 736)
    whole = rm.mxfp8_linear(x, w)
    for a, b in ((0, 129), (1000, 1300), (4000, 6000)):
        assert torch.equal(rm.mxfp8_linear(x[a:b].contiguous(), w), whole[a:b])


def test_shapes_of_the_product(rm):
    # leading dimensions are rows; a gate of [N] or [1, N] is every row's, one of [B, N] a batch's
    rng = np.random.default_rng(11)
    x = rows_of(rng, 24, 96, torch.float16).cuda()
    w, _ = make(rm, rng, 40, 96)
    g = torch.from_numpy(rng.standard_normal((2, 40))).half().cuda()
    flat = rm.mxfp8_linear(x, w, gate=g[0])
    for lead in ((24,), (2, 12), (2, 3, 4), (1, 24), (24, 1)):
        for gate in (g[0], g[:1], g[:1, None].expand(lead[0] if len(lead) > 1 else 1, 1, 40)):
            out = rm.mxfp8_linear(x.view(*lead, 96), w, gate=gate)
            assert out.shape == (*lead, 40) and torch.equal(out.view(24, 40), flat)
    out = rm.mxfp8_linear(x.view(2, 3, 4, 96), w, gate=g)
    assert torch.equal(out[0].view(12, 40), flat[:12])
    assert torch.equal(out[1].view(12, 40), rm.mxfp8_linear(x[12:].contiguous(), w, gate=g[1]))


@pytest.mark.parametrize("M", [70, 300])
def test_product_nan_stays_in_its_row(rm, M):
    rng = np.random.default_rng(4)
    x = rows_of(rng, M, 256, torch.bfloat16)
    x[3, 100] = float("inf")
    w, _ = make(rm, rng, 160, 256)
    out, kept = rm.mxfp8_linear(x.cuda(), w, activation="silu", keep=True)
    for bad in (torch.isnan(out), torch.isnan(rm.mxfp8_dequantize(kept))):
        assert bad[3].all() and not bad[:3].any() and not bad[4:].any()


@pytest.mark.parametrize("M", [5, 133])
def test_product_ignores_what_lies_behind_its_rows(rm, M):
    # NaN scales and any codes in the rows after the last one, and in the outputs behind it
    rng = np.random.default_rng(6)
    N, K = 32, 160
    a, av = make(rm, rng, M, K)
    b, bv = make(rm, rng, N, K)
    for q, rows in ((a, M), (b, N)):
        g = q.scales.view(-(-rows // 128), -1, 32, 4, 4)  # [.., tile, r % 32, r // 32, block]
        r = torch.arange(128, device="cuda").view(4, 32).T
        g[-1][(r >= (rows - 1) % 128 + 1).expand(g.shape[1], 32, 4)] = 255
    buf = torch.full((M + 3, N), 5.0, dtype=torch.bfloat16, device="cuda")
    c = torch.full((2, M + 3, N), 3.0, device="cuda").to(torch.float8_e4m3fn)
    s = torch.full((2, rm.mxfp8_scale_bytes(M, N) + 512,), 77, dtype=torch.uint8, device="cuda")
    n = rm.mxfp8_scale_bytes(M, N)
    rm.mxfp8_linear(a, b, out=buf[:M], keep=rm.Mxfp8(c[0, :M], s[0, :n]))
    rm.mxfp8_linear(a, b, out=rm.Mxfp8(c[1, :M], s[1, :n]), quantize=True)
    z = av @ bv.T
    slack = 8 * 2.0 ** -23 * (av.abs() @ bv.abs().T)
    assert (buf[M:] == 5.0).all() and (c[:, M:].float() == 3.0).all() and (s[:, n:] == 77).all()
    assert ((buf[:M].double() - z).abs() <= 2.0 ** -8 * z.abs() + slack).all()
    for i in range(2):
        _mx8.check_held(rm.Mxfp8(c[i, :M], s[i, :n]), z, slack)


def test_empty_product(rm):
    w, _ = make(rm, np.random.default_rng(1), 32, 64)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert rm.mxfp8_linear(x, w).shape == (0, 32)
    y, kept = rm.mxfp8_linear(x, w, quantize=True, keep=True)
    assert y.codes.shape == kept.codes.shape == (0, 32)


@pytest.mark.parametrize("M", [1, 32, 33, 200])
def test_product_added_to_its_own_rows(rm, M):
    x = torch.randn(M, 160, device="cuda").bfloat16()
    w = rm.mxfp8_quantize(torch.randn(160, 160, device="cuda").bfloat16())
    want = rm.mxfp8_linear(x, w, activation="silu", residual=x)
    plain = rm.mxfp8_linear(x, w)
    y = x.clone()
    assert rm.mxfp8_linear(y, w, activation="silu", residual=y, out=y) is y and torch.equal(y, want)
    y = x.clone()
    rm.mxfp8_linear(y, w, out=y)
    assert torch.equal(y, plain)
