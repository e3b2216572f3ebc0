"""The 8-bit gradients' sums over the tokens as sums of small integers, where nothing rounds: equal to sums
in 64 bits, so that one row lost or counted twice shows, however many there are.  Checkpoints, gradients
and statistics are small integers and ones; weights, gates and 1 + scale are powers of two."""
import pytest
import torch

from test_gpu_column_sums import Integers, equal

pytestmark = pytest.mark.gpu

# items of 128 rows by 128 columns and runs of rows: whole and not, fewer and more than the SMs take at once
SHAPES = [(1, 1, 32), (1, 21000, 512), (2, 9001, 4096), (3, 4097, 6144), (1, 100000, 64),
          (2, 2500, 16384), (160, 7, 1024), (400, 1, 4096), (40, 300, 1056), (1000, 1, 12288),
          (3000, 2, 256), (5, 128, 8192)]


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0
    torch.cuda.empty_cache()


def held(rm, t):
    """t in 8-bit blocks, which hold small integers as they are."""
    q = rm.mxfp8_quantize(t)
    assert torch.equal(rm.mxfp8_dequantize(q, dtype=t.dtype), t)
    return q


def check(rm, t, gate=None):
    wide = lambda v: v.double().view(-1, v.shape[-1])  # noqa: E731
    q = held(rm, t.x)
    plain, with_x = t.sums(t.go), t.sums(t.go, t.x)
    _, gw, gsc, gsh = rm.rmsnorm_mxfp8_backward(q, t.w, t.scale, t.go, t.stat, need_x=False)
    equal(gsh, t.over(plain))
    equal(gsc, t.over(with_x) * wide(t.w))
    equal(gw, (with_x * (1 + wide(t.scale))).sum(0))
    # without an activation z is the values themselves
    _, grad_bias, _ = rm.mxfp8_activation_backward(q, t.go)
    equal(grad_bias, plain.sum(0))
    _, grad_bias, grad_gate = rm.mxfp8_activation_backward(q, t.go, gate=t.gate)
    equal(grad_bias, (plain * wide(t.gate)).sum(0))
    equal(grad_gate, t.over(with_x))
    return with_x


@pytest.mark.parametrize("per_batch", [False, True])
@pytest.mark.parametrize("B,S,D", SHAPES)
def test_column_sums(rm, B, S, D, per_batch):
    check(rm, Integers(B, S, D, torch.bfloat16, per_batch))


def test_column_sums_fp16(rm):
    check(rm, Integers(2, 5000, 1536, torch.float16, True))


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("rows", [130, 9001, 40000])
def test_sums_of_an_activation_where_it_is_the_identity(rm, rows, act):
    # far from 0 an activation is its argument or 0, and its derivative 1 or 0, to the last bit
    t = Integers(1, rows, 160, torch.bfloat16, False)
    q = held(rm, t.x * 2.0 ** 10)
    z = t.x.double() * 2.0 ** 10
    on = (z > 0).double() + 0.5 * (z == 0)  # (the derivative at 0)
    _, grad_bias, grad_gate = rm.mxfp8_activation_backward(q, t.go, act, t.gate)
    equal(grad_bias * 2, 2 * (t.go.double() * on * t.gate.double()).sum((0, 1)))
    want = (t.go.double() * z.clamp(min=0.0)).sum((0, 1))
    equal(grad_gate[0] * 2.0 ** -10, want * 2.0 ** -10)
    _, grad_bias, _ = rm.mxfp8_activation_backward(q, t.go, act)
    equal(grad_bias * 2, 2 * (t.go.double() * on).sum((0, 1)))


def test_one_row_less_is_another_sum(rm):
    # what the equality above can tell: the sums without any one of some rows are others
    t = Integers(1, 9001, 512, torch.bfloat16, False)
    whole = check(rm, t)
    for row in (0, 4500, 9000):
        assert not torch.equal(whole, whole - t.go[:, row].double() * t.x[:, row].double())


def test_column_sums_past_32_bits(rm):
    check(rm, Integers(1, 140000, 16384, torch.bfloat16, False))  # 2.3e9 values
