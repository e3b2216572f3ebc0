"""Microscaled 8-bit operators without a GPU: the definition's own pins, sizes, and every refusal
(status codes and exceptions before anything is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import _mx8

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_STRIDE, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
P = ctypes.c_void_p
A = 0x10000000  # aligned addresses that nothing dereferences


def at(i):
    return A + (i << 26)


@pytest.fixture(scope="module")
def rm():
    from rmsnorm_modulate_gb300 import _build

    _build.build()
    import rmsnorm_modulate_gb300 as rm

    rm.library()
    return rm


def test_reference_blocks_by_hand():
    x = np.zeros((1, 32))
    x[0, :6] = [448.0, -448.0, 17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10]
    codes, e = _mx8.quantize(x)
    assert e[0, 0] == 127  # 448 fits under 2^0
    got = _mx8.values(codes, e)[0]
    # ties: 17 -> 16, 19 -> 20, half of the smallest code -> 0, one and a half -> two of it
    assert got[:6].tolist() == [448.0, -448.0, 16.0, 20.0, 0.0, 2.0 ** -8]
    x[0, 0] = 449.0  # the next power of two
    codes, e = _mx8.quantize(x)
    assert e[0, 0] == 128 and _mx8.values(codes, e)[0, 0] == 448.0
    x[0, 3] = np.inf
    assert _mx8.quantize(x)[1][0, 0] == 255
    assert _mx8.quantize(np.zeros((1, 32)))[1][0, 0] == 0
    assert _mx8.quantize(np.full((1, 32), 2.0 ** -140))[1][0, 0] == 0


def test_reference_codes_are_e4m3():
    # torch's own type: every value, and the rounding of values between
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(bits, _mx8.MAGS)
    v = np.random.default_rng(1).uniform(-448, 448, 4000) * np.exp2(
        np.random.default_rng(2).integers(-16, 1, 4000))
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    f32 = torch.from_numpy(v).float().double().numpy()  # torch rounds by way of fp32
    assert np.array_equal(_mx8.nearest(f32), want)


def test_reference_tiles_round_trip():
    g = np.random.default_rng(0).integers(0, 255, (300, 11)).astype(np.uint8)
    t = _mx8.tiles(g, 352)
    assert t.size == _mx8.scale_bytes(300, 352)
    assert np.array_equal(_mx8.grid(t, 300, 352), g)


def test_scale_bytes(rm):
    for rows, K in ((1, 32), (128, 128), (129, 160), (4216, 16384), (0, 64)):
        assert rm.mxfp8_scale_bytes(rows, K) == _mx8.scale_bytes(rows, K)
    for rows, K in ((1, 0), (1, 48), (-1, 32), (1 << 31, 32), (1, 1 << 21)):
        assert rm.mxfp8_scale_bytes(rows, K) == 0


def test_supported(rm):
    for op, good, bad in ((rm.OP_MXFP8, (32, 1 << 20), (48, 0, (1 << 20) + 32)),
                          (rm.OP_ADD_RMSNORM_MXFP8, (32, 16384), (40, 16416))):
        assert all(rm.supported(op, d) for d in good)
        assert not any(rm.supported(op, d) for d in bad)


def test_rows_refusals(rm):
    lib = rm.library()
    for name in ("mxfp8_quantize", "mxfp8_dequantize"):
        f = getattr(lib, name)

        def call(a=at(0), b=at(1), c=at(2), rows=4, K=64, dtype=0):
            return f(P(a), P(b), P(c), rows, K, dtype, P(0))

        assert call(K=48) == ERR_SHAPE and call(K=0) == ERR_SHAPE and call(rows=-1) == ERR_SHAPE
        assert call(K=(1 << 20) + 32) == ERR_SHAPE and call(rows=1 << 31) == ERR_SHAPE
        assert call(rows=1 << 24, K=1 << 20) == ERR_SHAPE  # more units than 32 bits count
        assert call(dtype=2) == ERR_UNSUPPORTED
        assert call(rows=0, a=0, b=0, c=0) == OK  # nothing to do
        for k in "abc":
            assert call(**{k: 0}) == ERR_NULL
            assert call(**{k: at(3) + 8}) == ERR_ALIGN
        assert call(b=at(0)) == ERR_UNSUPPORTED and call(c=at(0) + 64) == ERR_UNSUPPORTED
        assert call(c=at(1) + 64) == ERR_UNSUPPORTED


def test_transpose_refusals(rm):
    f = rm.library().mxfp8_transpose

    def call(a=at(0), b=at(1), c=at(2), d=at(3), rows=40, K=64):
        return f(P(a), P(b), P(c), P(d), rows, K, P(0))

    for k in (dict(K=48), dict(K=0), dict(rows=-1), dict(rows=(1 << 20) + 1),
              dict(K=(1 << 20) + 32)):
        assert call(**k) == ERR_SHAPE, k
    assert call(rows=0, a=0) == OK
    for k in "abcd":
        assert call(**{k: 0}) == ERR_NULL
        assert call(**{k: at(4) + 8}) == ERR_ALIGN
    # over an input or one another; the result of 40 rows has 64 bytes in each of its own
    for k in (dict(c=at(0)), dict(d=at(0) + 64), dict(c=at(1)), dict(d=at(2) + 4080),
              dict(c=at(1) - 4080)):
        assert call(**k) == ERR_UNSUPPORTED, k


def test_matmul_refusals(rm):
    f = rm.library().mxfp8_matmul

    def call(a=at(0), sa=at(1), b=at(2), sb=at(3), bias=at(4), act=1, gate=at(5), gs=0, res=at(6),
             out=at(7), so=at(8), keep=at(9), sk=at(10), B=2, S=100, N=128, K=64, dtype=0):
        return f(P(a), P(sa), P(b), P(sb), P(bias), act, P(gate), gs, P(res), P(out), P(so), P(keep),
                 P(sk), B, S, N, K, dtype, P(0))

    for k in (dict(N=12), dict(N=-8), dict(B=-1), dict(S=-1), dict(K=40), dict(K=0), dict(N=136),
              dict(N=72, keep=0, sk=0), dict(N=72, so=0), dict(B=1 << 40, S=1 << 40),
              dict(N=(1 << 23) + 32), dict(S=1 << 31)):
        assert call(**k) == ERR_SHAPE, k
    assert call(dtype=7) == ERR_UNSUPPORTED and call(dtype=-1) == ERR_UNSUPPORTED
    assert call(act=4) == ERR_UNSUPPORTED and call(act=-1) == ERR_UNSUPPORTED
    assert call(gs=4) == ERR_STRIDE and call(gs=-8) == ERR_STRIDE
    for k in ("a", "b", "sb", "out", "keep", "sk"):
        assert call(**{k: 0}) == ERR_NULL, k
    # rows that the call quantises: few, and 16 bits wide
    assert call(sa=0, S=17) == ERR_SHAPE and call(sa=0, S=2, dtype=2) == ERR_UNSUPPORTED
    assert call(sa=0, S=2, out=at(0) + 4 * 64) == ERR_UNSUPPORTED  # over the second half of a
    for k in ("a", "sa", "b", "sb", "bias", "gate", "res", "out", "so", "keep", "sk"):
        assert call(**{k: at(11) + 8}) == ERR_ALIGN, k
    assert call(S=0, a=0) == OK and call(N=0, a=0) == OK
    for to in ("out", "so", "keep", "sk"):
        for k in range(7):
            if to != "out" or k != 6:
                assert call(**{to: at(k)}) == ERR_UNSUPPORTED, (to, k)
    for k in (dict(keep=at(7)), dict(sk=at(8)), dict(so=at(7) + 128), dict(sk=at(9) + 128)):
        assert call(**k) == ERR_UNSUPPORTED, k
    assert call(out=at(6)) == ERR_UNSUPPORTED  # an 8-bit result in the residual's place
    assert call(out=at(6) + 16, so=0) == ERR_UNSUPPORTED  # residual shifted by a vector
    assert call(gate=at(7) - 2 * 1024, gs=1024) == ERR_UNSUPPORTED  # the second gate row
    # an fp32 result and its gate rows reach twice as far
    assert call(out=at(6) - 2 * 100 * 128 * 4 + 64, so=0, dtype=2) == ERR_UNSUPPORTED
    assert call(gate=at(7) - 4 * 1024, gs=1024, dtype=2) == ERR_UNSUPPORTED


def test_norm_refusals(rm):
    f = rm.library().add_rmsnorm_mxfp8

    def call(x=at(0), u=at(1), w=at(2), sc=at(3), sh=at(4), bs=0, res=at(5), out=at(6), so=at(7),
             keep=at(8), sk=at(9), B=2, S=50, D=64, rstd=at(10), dtype=0):
        return f(P(x), P(u), P(w), P(sc), P(sh), bs, P(res), P(out), P(so), P(keep), P(sk), B, S, D,
                 1e-6, P(rstd), dtype, P(0))

    for k in (dict(D=40), dict(D=0), dict(D=16416), dict(B=-1), dict(S=-1), dict(S=1 << 31)):
        assert call(**k) == ERR_SHAPE, k
    assert call(dtype=2) == ERR_UNSUPPORTED
    assert call(bs=4) == ERR_STRIDE and call(bs=-8) == ERR_STRIDE
    assert call(S=0, x=0) == OK
    for k in ("x", "res", "out", "so", "keep", "sk"):
        assert call(**{k: 0}) == ERR_NULL, k
    assert call(u=0) == ERR_UNSUPPORTED  # a place for the sum without a sum
    for k in ("x", "u", "w", "sc", "sh", "res", "out", "so", "keep", "sk"):
        assert call(**{k: at(11) + 8}) == ERR_ALIGN, k
    assert call(rstd=at(10) + 2) == ERR_ALIGN
    for to in ("out", "so", "keep", "sk", "rstd"):
        for k in range(10):
            if at(k) != dict(out=at(6), so=at(7), keep=at(8), sk=at(9), rstd=0)[to]:
                assert call(**{to: at(k)}) == ERR_UNSUPPORTED, (to, k)
    for k in (0, 1):  # the sum may take a row tensor's place, not a part of it
        assert call(res=at(k) + 16) == ERR_UNSUPPORTED
    for k in (2, 3, 4, 6, 7, 8, 9, 10):
        assert call(res=at(k)) == ERR_UNSUPPORTED, k


def test_norm_backward_refusals(rm):
    f, ws = rm.library().rmsnorm_mxfp8_backward, rm.library().rmsnorm_mxfp8_backward_workspace_bytes
    assert ws(0, 4, 64) == 0 and ws(1, 0, 64) == 0 and ws(1, 4, 48) == 0
    assert ws(2, 50, 64) >= 2 * 2 * 64 * 4

    def call(k=at(0), sk=at(1), w=at(2), sc=at(3), bs=0, go=at(4), gr=at(5), rstd=at(6), B=2, S=50,
             D=64, gx=at(7), gw=at(8), gs=at(9), gh=at(10), work=at(11), wb=1 << 24, dtype=0):
        return f(P(k), P(sk), P(w), P(sc), bs, P(go), P(gr), P(rstd), B, S, D, P(gx), P(gw), P(gs),
                 P(gh), P(work), wb, dtype, P(0))

    for k in (dict(D=40), dict(D=16416), dict(B=-1), dict(S=-1), dict(S=1 << 31), dict(wb=64)):
        assert call(**k) == ERR_SHAPE, k
    assert call(dtype=2) == ERR_UNSUPPORTED and call(bs=4) == ERR_STRIDE
    for k in ("k", "sk", "go", "rstd", "work"):
        assert call(**{k: 0}) == ERR_NULL, k
    for k in ("k", "sk", "w", "sc", "go", "gr", "gx", "gw", "gs", "gh"):
        assert call(**{k: at(12) + 8}) == ERR_ALIGN, k
    assert call(work=at(11) + 16) == ERR_ALIGN and call(rstd=at(6) + 2) == ERR_ALIGN
    assert call(gx=0, gw=0, gs=0, gh=0) == OK  # nothing wanted
    for to, own in (("gx", 7), ("gw", 8), ("gs", 9), ("gh", 10), ("work", 11)):
        for k in range(12):
            if k != own:
                assert call(**{to: at(k)}) == ERR_UNSUPPORTED, (to, k)


def test_activation_backward_refusals(rm):
    f = rm.library().mxfp8_activation_backward
    ws = rm.library().mxfp8_activation_backward_workspace_bytes
    assert ws(0, 4, 64) == 0 and ws(1, 0, 64) == 0 and ws(1, 4, 48) == 0
    assert ws(2, 130, 64) >= 2 * 2 * 2 * 64 * 4

    def call(z=at(0), sz=at(1), go=at(2), act=1, gate=at(3), gs=0, dz=at(4), sd=at(5), gb=at(6),
             gg=at(7), B=2, S=50, N=64, work=at(8), wb=1 << 24, dtype=0):
        return f(P(z), P(sz), P(go), act, P(gate), gs, P(dz), P(sd), P(gb), P(gg), B, S, N, P(work),
                 wb, dtype, P(0))

    for k in (dict(N=40), dict(N=0), dict(B=-1), dict(S=-1), dict(S=1 << 31), dict(wb=64),
              dict(B=1 << 40, S=1 << 40)):
        assert call(**k) == ERR_SHAPE, k
    assert call(dtype=2) == ERR_UNSUPPORTED and call(act=4) == ERR_UNSUPPORTED
    assert call(gate=0) == ERR_UNSUPPORTED  # a gradient by something that took no part
    assert call(gs=4) == ERR_STRIDE
    for k in ("z", "sz", "go", "dz", "sd", "work"):
        assert call(**{k: 0}) == ERR_NULL, k
    for k in ("z", "sz", "go", "gate", "dz", "sd", "gb", "gg"):
        assert call(**{k: at(9) + 8}) == ERR_ALIGN, k
    assert call(work=at(8) + 16) == ERR_ALIGN
    for to, own in (("dz", 4), ("sd", 5), ("gb", 6), ("gg", 7), ("work", 8)):
        for k in range(9):
            if k != own:
                assert call(**{to: at(k)}) == ERR_UNSUPPORTED, (to, k)


def test_python_refusals(rm):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = rm.Mxfp8(torch.zeros(4, 64, dtype=torch.uint8).view(torch.float8_e4m3fn),
                 torch.zeros(512, dtype=torch.uint8))
    for call in (lambda: rm.mxfp8_quantize(x), lambda: rm.mxfp8_dequantize(q),
                 lambda: rm.mxfp8_transpose(q), lambda: rm.mxfp8_linear(x, q),
                 lambda: rm.add_rmsnorm_mxfp8(x), lambda: rm.mxfp8_activation_backward(q, x),
                 lambda: rm.rmsnorm_mxfp8_backward(q, None, None, x, torch.zeros(4))):
        with pytest.raises(ValueError):  # no CPU path
            call()
    for call in (lambda: rm.mxfp8_quantize(x.float()), lambda: rm.mxfp8_quantize([1.0]),
                 lambda: rm.mxfp8_dequantize(x), lambda: rm.mxfp8_transpose(x),
                 lambda: rm.mxfp8_linear(q, q, dtype=torch.float64),
                 lambda: rm.mxfp8_activation_backward(x, x),
                 lambda: rm.rmsnorm_mxfp8_backward(x, None, None, x, None),
                 lambda: rm.add_rmsnorm_mxfp8(x.double())):
        with pytest.raises(TypeError):
            call()
