"""Microscaled 4-bit operators without a GPU: the reference's own pins, sizes, and every refusal
(status codes and exceptions before anything is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import _mx

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_STRIDE, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
P = ctypes.c_void_p
A = 0x10000000  # aligned addresses that nothing dereferences


@pytest.fixture(scope="module")
def rm():
    from rmsnorm_modulate_gb300 import _build

    _build.build()
    import rmsnorm_modulate_gb300 as rm

    rm.library()
    return rm


def test_reference_blocks_by_hand():
    x = np.zeros((1, 32))
    x[0, :8] = [6.0, -6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 5.0]
    codes, e = _mx.quantize(x)
    assert e[0, 0] == 127  # 6 fits under 2^0
    # ties: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 5 -> 4
    assert codes[0, :8].tolist() == [7, 15, 0, 2, 2, 4, 4, 6]
    x[0, 0] = 6.0625  # the next power of two
    codes, e = _mx.quantize(x)
    assert e[0, 0] == 128 and codes[0, 0] == 5  # 3.03 -> 3
    x[0, 3] = np.inf
    assert _mx.quantize(x)[1][0, 0] == 255
    assert _mx.quantize(np.zeros((1, 32)))[1][0, 0] == 0


def test_reference_tiles_round_trip():
    g = np.random.default_rng(0).integers(0, 255, (300, 11)).astype(np.uint8)
    t = _mx.tiles(g, 352)
    assert t.size == _mx.scale_bytes(300, 352)
    assert np.array_equal(_mx.grid(t, 300, 352), g)


def test_scale_bytes(rm):
    for rows, K in ((1, 32), (128, 128), (129, 160), (4216, 16384), (0, 64)):
        assert rm.mxfp4_scale_bytes(rows, K) == _mx.scale_bytes(rows, K)
    for rows, K in ((1, 0), (1, 48), (-1, 32), (1 << 31, 32), (1, 1 << 21)):
        assert rm.mxfp4_scale_bytes(rows, K) == 0


def test_rows_refusals(rm):
    lib = rm.library()
    for name in ("mxfp4_quantize", "mxfp4_dequantize"):
        f = getattr(lib, name)

        def call(a=A, b=A + (1 << 24), c=A + (2 << 24), rows=4, K=64, dtype=0):
            return f(P(a), P(b), P(c), rows, K, dtype, P(0))

        assert call(K=48) == ERR_SHAPE and call(K=0) == ERR_SHAPE and call(rows=-1) == ERR_SHAPE
        assert call(K=(1 << 20) + 32) == ERR_SHAPE and call(rows=1 << 31) == ERR_SHAPE
        assert call(rows=1 << 24, K=1 << 20) == ERR_SHAPE  # more units than 32 bits count
        assert call(dtype=2) == ERR_UNSUPPORTED
        assert call(rows=0, a=0, b=0, c=0) == OK  # nothing to do
        for k in "abc":
            assert call(**{k: 0}) == ERR_NULL
            assert call(**{k: A + (3 << 24) + 8}) == ERR_ALIGN
        assert call(b=A) == ERR_UNSUPPORTED  # the outputs overlap an input, or one another
        assert call(c=A + 64) == ERR_UNSUPPORTED
        assert call(c=A + (1 << 24) + 64) == ERR_UNSUPPORTED


def test_matmul_refusals(rm):
    f = rm.library().mxfp4_matmul
    at = lambda i: A + (i << 26)  # noqa: E731

    def call(a=at(0), sa=at(1), b=at(2), sb=at(3), bias=at(4), gate=at(5), gs=0, res=at(6),
             out=at(7), B=2, S=100, N=128, K=64, dtype=0):
        return f(P(a), P(sa), P(b), P(sb), P(bias), P(gate), gs, P(res), P(out), B, S, N, K, dtype,
                 P(0))

    for k in (dict(N=12), dict(N=-8), dict(B=-1), dict(S=-1), dict(K=40), dict(K=0),
              dict(B=1 << 40, S=1 << 40), dict(N=(1 << 23) + 8), dict(S=1 << 31)):
        assert call(**k) == ERR_SHAPE, k
    assert call(dtype=7) == ERR_UNSUPPORTED
    assert call(gs=4) == ERR_STRIDE and call(gs=-8) == ERR_STRIDE
    for k in ("a", "sa", "b", "sb", "out"):
        assert call(**{k: 0}) == ERR_NULL, k
    for k in ("a", "sa", "b", "sb", "bias", "gate", "res", "out"):
        assert call(**{k: at(8) + 8}) == ERR_ALIGN, k
    assert call(S=0, a=0) == OK and call(N=0, a=0) == OK
    for k in (0, 1, 2, 3, 4, 5):
        assert call(out=at(k)) == ERR_UNSUPPORTED, k
    assert call(out=at(6) + 16) == ERR_UNSUPPORTED  # residual shifted by a vector
    assert call(gate=at(7) - 2 * 1024, gs=1024) == ERR_UNSUPPORTED  # the second gate row


def test_python_refusals(rm):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rm.mxfp4_quantize(x)  # no CPU path
    with pytest.raises(TypeError):
        rm.mxfp4_quantize(x.float())
    with pytest.raises(TypeError):
        rm.mxfp4_quantize([1.0])
    with pytest.raises(TypeError):
        rm.mxfp4_dequantize(x)
    q = rm.Mxfp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(ValueError):
        rm.mxfp4_dequantize(q)
    with pytest.raises(ValueError):
        rm.mxfp4_linear(x, q)
    with pytest.raises(TypeError):
        rm.mxfp4_linear(q, q, dtype=torch.float32)
