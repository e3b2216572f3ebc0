"""The microscaled 4-bit operators against their definition in 64 bits.

Quantisation is exact (power-of-two scales, one rounding to a code), so codes and scale bytes are
compared for equality.  The product's bound per element is the output's half step, eps / 2 of the
result, and of its fp32 accumulation: every step of 64 values adds to the running sum with an
error of at most 2^-23 (a truncation) of the magnitudes summed, and the epilogue's three
operations with 2^-24 of theirs."""
import numpy as np
import pytest
import torch

import _mx

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


def check_blocks(rm, x):
    rows, K = x.shape
    q = rm.mxfp4_quantize(x.cuda())
    y = rm.mxfp4_dequantize(q, dtype=x.dtype)
    codes, e = _mx.quantize(x.double().numpy())
    got = q.packed.cpu().numpy()
    fine = np.repeat(e != 255, 16, axis=1)
    assert np.array_equal(got[fine], _mx.pack(codes)[fine])
    assert np.array_equal(q.scales.cpu().numpy(), _mx.tiles(e, K))  # the padding's zeros too
    want = torch.from_numpy(_mx.values(got, e)).to(x.dtype)
    assert torch.equal(torch.nan_to_num(y.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))
    return q


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,K", [(1, 32), (3, 64), (127, 96), (128, 128), (129, 160), (33, 4128),
                                    (257, 1056), (640, 512)])
def test_quantize(rm, rows, K, dtype):
    check_blocks(rm, rows_of(np.random.default_rng(rows + K), rows, K, dtype))


@pytest.mark.parametrize("dtype", TYPES)
def test_quantize_edges(rm, dtype):
    f = torch.finfo(dtype)
    x = torch.zeros(12, 64, dtype=dtype)
    x[1, 0], x[1, 40] = f.max, -f.max
    x[2, 0] = f.smallest_normal
    x[3, 5] = f.smallest_normal * f.eps  # the smallest subnormal
    x[4, 0] = float("nan")
    x[5, 33] = float("inf")
    x[6, 0] = -float("inf")
    x[7] = torch.arange(64) / 4 - 6  # every tie of the grid
    x[8] = -0.0
    x[9, 0], x[9, 1] = 6.0, 3.0
    x[10, 0], x[10, 1] = 6.0 * (1 + f.eps), 3.0  # one step past the border
    x[11, 0], x[11, 1] = 1.5, f.max
    check_blocks(rm, x)


def test_quantize_every_bf16(rm):
    # each finite pattern against a block that keeps the scale at 2^0, then alone
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    alone = torch.zeros(1 << 11, 32, dtype=torch.bfloat16)
    alone[:, 0] = bits[::32]
    check_blocks(rm, alone)
    small = bits[bits.abs() <= 6]
    x = torch.full((-(-small.numel() // 31), 32), 6.0, dtype=torch.bfloat16)
    flat = torch.zeros(x.shape[0] * 31, dtype=torch.bfloat16)
    flat[:small.numel()] = small
    x[:, 1:] = flat.view(-1, 31)
    check_blocks(rm, x)


def test_quantize_leading_shape_and_empty(rm):
    x = rows_of(np.random.default_rng(5), 6, 64, torch.bfloat16)
    a, b = rm.mxfp4_quantize(x.view(2, 3, 64).cuda()), rm.mxfp4_quantize(x.cuda())
    assert a.packed.shape == (2, 3, 32)
    assert torch.equal(a.packed.view(6, 32), b.packed) and torch.equal(a.scales, b.scales)
    assert rm.mxfp4_dequantize(a).shape == (2, 3, 64)
    q = rm.mxfp4_quantize(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"))
    assert q.packed.shape == (0, 32) and q.scales.numel() == 0
    assert rm.mxfp4_dequantize(q).shape == (0, 64)


def make(rm, rng, rows, K):
    """A random 4-bit matrix, codes and scales alike, and its values."""
    packed = rng.integers(0, 256, (rows, K // 2)).astype(np.uint8)
    e = rng.integers(118, 130, (rows, K // 32)).astype(np.uint8)
    q = rm.Mxfp4(torch.from_numpy(packed).cuda(), torch.from_numpy(_mx.tiles(e, K)).cuda())
    return q, torch.from_numpy(_mx.values(packed, e)).cuda()


def check_product(rm, rng, B, S, N, K, dtype, bias=False, gate=None, residual=False, inplace=False):
    a, av = make(rm, rng, B * S, K)
    b, bv = make(rm, rng, N, K)
    half = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype).cuda()  # noqa: E731
    bt = half(N) if bias else None
    gt = None
    if gate:  # a view into rows of three, as an adaLN projection gives it
        gt = half(B if gate == "batch" else 1, 1, 3 * N).chunk(3, -1)[1]
    rt = half(B, S, N) * 8 if residual else None
    want, size = av @ bv.T, av.abs() @ bv.abs().T
    slack = (K / 64 + 2) * 2.0 ** -23 * size
    want, size, slack = (t.view(B, S, N) for t in (want, size, slack))
    if bias:
        want, size = want + bt.double(), size + bt.double().abs()
    if gate:
        want, size, slack = (want * gt.double(), size * gt.double().abs(),
                             slack * gt.double().abs())
    if residual:
        want, size = want + rt.double(), size + rt.double().abs()
    q = rm.Mxfp4(a.packed.view(B, S, K // 2), a.scales)
    out = rm.mxfp4_linear(q, b, bias=bt, gate=gt, residual=rt, dtype=dtype,
                          out=rt if inplace else None)
    assert out.shape == (B, S, N) and out.dtype == dtype
    f = torch.finfo(dtype)
    over = want.abs() > float(f.max)
    bound = f.eps / 2 * want.abs() + slack + 3 * 2.0 ** -24 * size + f.smallest_normal * f.eps
    off = ((out.double() - want).abs() / bound)[~over]
    assert not off.numel() or off.max().item() <= 1.0, (B, S, N, K, off.max().item())
    return out


@pytest.mark.parametrize("M,N,K", [
    (1, 8, 32), (1, 4096, 64), (5, 264, 96), (8, 1000, 4096), (16, 128, 2080), (127, 256, 128),
    (128, 256, 256), (129, 248, 288), (200, 520, 1056), (640, 1536, 512), (1000, 3080, 736),
    (33, 72, 16384),
])
@pytest.mark.parametrize("dtype", TYPES)
def test_product(rm, M, N, K, dtype):
    check_product(rm, np.random.default_rng(M + N + K), 1, M, N, K, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,S,N,K,kw", [
    (1, 7, 264, 512, dict(bias=True)),
    (3, 50, 136, 320, dict(gate="batch", residual=True)),
    (2, 129, 512, 1024, dict(bias=True, gate="shared", residual=True)),
    (2, 1, 4096, 256, dict(bias=True, gate="batch", residual=True, inplace=True)),
    (4, 33, 40, 64, dict(gate="batch")),
    (1, 300, 280, 2048, dict(residual=True, inplace=True)),
])
def test_product_epilogue(rm, B, S, N, K, kw, dtype):
    check_product(rm, np.random.default_rng(B * S + N), B, S, N, K, dtype, **kw)


def test_product_of_integers_is_exact(rm):
    # codes whose products and sums are small integers: no rounding anywhere
    rng = np.random.default_rng(3)
    ints = np.array([0, 2, 4, 5, 6, 7, 10, 12, 13, 14, 15])  # 0, 1, 2, 3, 4, 6 and their negatives
    for M, N, K in ((40, 72, 32), (130, 264, 160), (8, 512, 512)):
        e = {}
        q = {}
        for name, rows in (("a", M), ("b", N)):
            codes = ints[rng.integers(0, len(ints), (rows, K))].astype(np.uint8)
            codes[rng.random((rows, K)) < 0.8] = 0
            grid = np.full((rows, K // 32), 127, np.uint8)
            e[name] = _mx.values(_mx.pack(codes), grid)
            q[name] = rm.Mxfp4(torch.from_numpy(_mx.pack(codes)).cuda(),
                               torch.from_numpy(_mx.tiles(grid, K)).cuda())
        out = rm.mxfp4_linear(q["a"], q["b"], dtype=torch.float16)
        want = e["a"] @ e["b"].T
        assert np.abs(want).max() < 2048
        assert np.array_equal(out.double().cpu().numpy(), want)


def test_product_quantises_its_rows(rm):
    rng = np.random.default_rng(9)
    x = rows_of(rng, 77, 608, torch.bfloat16).cuda()
    w, _ = make(rm, rng, 264, 608)
    a = rm.mxfp4_linear(x, w)
    assert torch.equal(a, rm.mxfp4_linear(rm.mxfp4_quantize(x), w))
    # a row's result does not depend on the rows beside it
    b = rm.mxfp4_linear(x[5:9].contiguous(), w)
    assert torch.equal(a[5:9], b)


def test_shapes_of_the_product(rm):
    # leading dimensions are rows; a gate of [N] or [1, N] is every row's, one of [B, N] a batch's
    rng = np.random.default_rng(11)
    x = rows_of(rng, 24, 96, torch.float16).cuda()
    w, _ = make(rm, rng, 40, 96)
    g = torch.from_numpy(rng.standard_normal((2, 40))).half().cuda()
    flat = rm.mxfp4_linear(x, w, gate=g[0])
    for lead in ((24,), (2, 12), (2, 3, 4), (1, 24), (24, 1)):
        for gate in (g[0], g[:1], g[:1, None].expand(lead[0] if len(lead) > 1 else 1, 1, 40)):
            out = rm.mxfp4_linear(x.view(*lead, 96), w, gate=gate)
            assert out.shape == (*lead, 40) and torch.equal(out.view(24, 40), flat)
    out = rm.mxfp4_linear(x.view(2, 3, 4, 96), w, gate=g)
    assert torch.equal(out[0].view(12, 40), flat[:12])
    assert torch.equal(out[1].view(12, 40), rm.mxfp4_linear(x[12:].contiguous(), w, gate=g[1]))


def test_rows_do_not_depend_on_how_many_there_are(rm):
    # past 128 rows: narrow and wide tiles give a row the same bits
    rng = np.random.default_rng(10)
    x = rows_of(rng, 6000, 736, torch.bfloat16).cuda()
    w, _ = make(rm, rng, 2056, 736)
    whole = rm.mxfp4_linear(x, w)
    for a, b in ((0, 129), (1000, 1300), (4000, 6000)):
        assert torch.equal(rm.mxfp4_linear(x[a:b].contiguous(), w), whole[a:b])


def test_product_nan_scale_stays_in_its_row(rm):
    rng = np.random.default_rng(4)
    x = rows_of(rng, 70, 256, torch.bfloat16)
    x[3, 100] = float("inf")
    w, _ = make(rm, rng, 136, 256)
    out = rm.mxfp4_linear(x.cuda(), w)
    bad = torch.isnan(out)
    assert bad[3].all() and not bad[:3].any() and not bad[4:].any()


def test_product_ignores_what_lies_behind_its_rows(rm):
    # NaN scales and any codes in the rows after the last one, and in the output behind it
    rng = np.random.default_rng(6)
    M, N, K = 5, 24, 160
    a, av = make(rm, rng, M, K)
    b, bv = make(rm, rng, N, K)
    for q, rows in ((a, M), (b, N)):
        g = q.scales.view(-1, 32, 4, 4)  # [tile, r % 32, r // 32, block]
        r = torch.arange(128, device="cuda").view(4, 32).T
        g[(r >= rows).expand(g.shape[0], 32, 4)] = 255
    buf = torch.full((M + 3, N), 5.0, dtype=torch.bfloat16, device="cuda")
    rm.mxfp4_linear(a, b, out=buf[:M])
    want = av @ bv.T
    assert (buf[M:] == 5.0).all()
    bound = 2.0 ** -8 * want.abs() + 8 * 2.0 ** -23 * (av.abs() @ bv.abs().T)
    assert ((buf[:M].double() - want).abs() <= bound).all()


def test_empty_product(rm):
    w, _ = make(rm, np.random.default_rng(1), 16, 64)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert rm.mxfp4_linear(x, w).shape == (0, 16)


def test_streams_and_graph(rm):
    rng = np.random.default_rng(12)
    x = rows_of(rng, 100, 512, torch.bfloat16).cuda()
    w, _ = make(rm, rng, 520, 512)
    want = rm.mxfp4_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [rm.mxfp4_linear(x, w, stream=s) for _ in range(20)]
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(g, want) for g in got)
    g = torch.cuda.CUDAGraph()
    static = x.clone()
    with torch.cuda.graph(g):
        out = rm.mxfp4_linear(static, w)
    static.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want.flip(0))


def test_gpu_refusals(rm):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    w = rm.mxfp4_quantize(torch.zeros(16, 64, dtype=torch.bfloat16, device="cuda"))
    n = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    for bad in (n(4, 48), n(64, 4).t(), n(0)):
        with pytest.raises(ValueError):
            rm.mxfp4_quantize(bad)
    for kw in (dict(bias=n(8)), dict(gate=n(3, 1, 16)), dict(residual=n(4, 8)), dict(out=n(4, 8)),
               dict(bias=torch.zeros(16, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            rm.mxfp4_linear(x, w, **kw)
    for kw in (dict(bias=n(16, t=torch.float16)), dict(dtype=torch.float16)):
        with pytest.raises(TypeError):
            rm.mxfp4_linear(x, w, **kw)
    with pytest.raises(ValueError):
        rm.mxfp4_linear(n(4, 96), w)
    with pytest.raises(ValueError):  # too few scale bytes
        rm.mxfp4_linear(x, rm.Mxfp4(w.packed, w.scales[:256]))
    with pytest.raises(ValueError):  # 12 columns
        rm.mxfp4_linear(x, rm.mxfp4_quantize(n(12, 64)))
    with pytest.raises(rm.RmsmodError):  # rows that start between two 16-byte vectors
        rm.mxfp4_quantize(n(4 * 64 + 4)[4:].view(4, 64))
    with pytest.raises(rm.RmsmodError):  # the result over a part of the residual
        buf = n(5, 16)
        rm.mxfp4_linear(x, w, residual=buf[:4], out=buf[1:])
