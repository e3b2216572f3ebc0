"""The gradients of the row vectors as sums of small integers, where nothing rounds: equal to sums in
64 bits, so that one row lost or counted twice shows, however many there are.  Statistics are the
caller's, and ones here; weights, gates and 1 + scale are powers of two."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 8), (1, 21000, 512), (2, 9001, 4096), (3, 4097, 6144), (1, 100000, 64),
          (2, 2500, 16384), (160, 7, 1024), (400, 1, 4096), (40, 300, 1032), (1000, 1, 12288)]


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0
    torch.cuda.empty_cache()


class Integers:
    def __init__(self, B, S, D, dtype, per_batch):
        self.gen = torch.Generator(device="cuda").manual_seed(B + S + D)
        self.dtype, self.rows = dtype, B if per_batch else 1
        self.x, self.go = self.ints(B, S, D), self.ints(B, S, D)
        self.w, self.gate, one = self.powers(D), self.powers(self.rows, 1, D), \
            self.powers(self.rows, 1, D)
        self.scale = one - 1
        self.stat = torch.ones(B * S, device="cuda")

    def ints(self, *shape):
        return torch.randint(-2, 3, shape, device="cuda", generator=self.gen,
                             dtype=torch.int8).to(self.dtype)

    def powers(self, *shape):
        return torch.randint(0, 2, shape, device="cuda", generator=self.gen).add(1).to(self.dtype)

    def sums(self, first, second=None):
        """[B, D] sums over the tokens in 64 bits, some rows at a time."""
        B, S, D = first.shape
        total = torch.zeros(B, D, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 27) // (B * D))
        for i in range(0, S, step):
            t = first[:, i:i + step].double()
            total += (t if second is None else t * second[:, i:i + step].double()).sum(1)
        return total

    def over(self, t):
        return t if self.rows == t.shape[0] else t.sum(0, keepdim=True)


def equal(got, want):
    assert float(want.abs().max()) < 2 ** 24  # held exactly in fp32, as is every part of the sum
    assert torch.equal(got.double(), want)


def check(rm, t):
    wide = lambda v: v.double().view(-1, v.shape[-1])  # noqa: E731
    plain, with_x = t.sums(t.go), t.sums(t.go, t.x)
    sums = dict(shift=t.over(plain), scale=t.over(with_x) * wide(t.w),
                weight=(with_x * (1 + wide(t.scale))).sum(0))
    if t.dtype is torch.bfloat16:  # the only type of rmsnorm_modulate
        _, gw, gsc, gsh = rm.rmsnorm_modulate_backward(t.x, t.w, t.scale, t.go, t.stat, need_x=False)
        for got, name in ((gw, "weight"), (gsc, "scale"), (gsh, "shift")):
            equal(got, sums[name])
    g = rm.sandwich_rmsnorm_modulate_backward(t.x, t.x, t.w, t.gate, t.w, t.scale, None, t.go,
                                              t.stat, t.stat, need_x=False)
    for name in sums:
        equal(getattr(g, name), sums[name])
    # without the second norm dh is the stream's gradient itself
    g = rm.sandwich_rmsnorm_modulate_backward(t.x, None, t.w, t.gate, None, None, t.go, None, t.stat,
                                              None, need_x=False, update_scale=0.5)
    equal(g.gate, t.over(with_x) * wide(t.w) * 0.5)
    equal(g.post_weight, (with_x * wide(t.gate)).sum(0) * 0.5)
    return with_x


@pytest.mark.parametrize("per_batch", [False, True])
@pytest.mark.parametrize("B,S,D", SHAPES)
def test_column_sums(rm, B, S, D, per_batch):
    check(rm, Integers(B, S, D, torch.bfloat16, per_batch))


def test_column_sums_fp16(rm):
    check(rm, Integers(2, 5000, 1536, torch.float16, True))


def test_one_row_less_is_another_sum(rm):
    # what the equality above can tell: the sums without any one of some rows are others
    t = Integers(1, 9001, 512, torch.bfloat16, False)
    whole = check(rm, t)
    for row in (0, 4500, 9000):
        assert not torch.equal(whole, whole - t.go[:, row].double() * t.x[:, row].double())


def test_column_sums_past_32_bits(rm):
    check(rm, Integers(1, 140000, 16384, torch.bfloat16, False))  # 2.3e9 values
