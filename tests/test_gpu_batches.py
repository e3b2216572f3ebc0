"""The sandwich norms and their gradients for many batches of few rows: a CTA takes several items there
and changes batch between them (two CTAs at once past 8192 values, while the next batch's first row is
under way), and the column sums go over the batches in several passes.  Against the definition in
float64, within the bounds that _sandwich_chain counts."""
import pytest
import torch

import _sandwich as ref
import _sandwich_chain as chain

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


def close(got, want, size, steps, what):
    f = torch.finfo(got.dtype)
    half = 0.0 if got.dtype == torch.float32 else f.eps / 2
    # (a result below the type's normal values is off by half of the smallest one's step)
    bound = half * want.abs() + steps * U * size + f.smallest_normal * f.eps
    assert got.isfinite().all(), what
    worst = ((got.double() - want).abs() / bound).max().item()
    assert worst <= 1.0, f"{what}: {worst} times its bound"


class Boundary:
    def __init__(self, rm, B, S, D, dtype, per_batch):
        gen = torch.Generator(device="cuda").manual_seed(B + 3 * S + 5 * D)
        n = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.B, self.S, self.D, self.rows = B, S, D, B if per_batch else 1
        self.x, self.u, self.go, self.gr = (n(B, S, D).to(dtype) for _ in range(4))
        self.gate, self.scale, self.shift = (0.3 * n(self.rows, 1, 3 * D)).to(dtype).chunk(3, -1)
        self.w, self.pw = ((1 + 0.1 * n(D)).to(dtype) for _ in range(2))
        self.rp, self.r = (torch.empty(B * S, device="cuda") for _ in range(2))
        self.res, self.out = rm.sandwich_rmsnorm_modulate(
            self.x, self.u, self.pw, self.gate, self.w, self.scale, self.shift, residual_scale=0.5,
            update_scale=1.5, post_rstd_out=self.rp, rstd_out=self.r)

    def stat(self, t):
        return t.double().view(self.B, self.S, 1)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("per_batch", [False, True])
@pytest.mark.parametrize("B,S,D", [(160, 1, 4096), (400, 3, 1024), (1000, 1, 200), (153, 40, 520),
                                   (77, 5, 12288), (160, 1, 12288), (400, 2, 8200)])
def test_forward(rm, B, S, D, per_batch, dtype):
    t = Boundary(rm, B, S, D, dtype, per_batch)
    close(t.res, *ref.residual_add(t.x, t.u, t.pw, t.gate, 1e-6, 0.5, 1.5), chain.VALUE, "res")
    close(t.out, *ref.norm(t.res, t.w, t.scale, t.shift, 1e-6), chain.VALUE, "out")
    for got, of in ((t.rp, t.u), (t.r, t.res)):
        want = ref.rstd(of, 1e-6).view(-1)
        close(got, want, want, chain.VALUE, "statistics")


def check_columns(t, got, want, names):
    for name in names:
        shared = t.rows == 1 or "weight" in name
        steps = chain.TERM + 4 + chain.column_additions(t.B, t.S, t.D, shared)
        x = getattr(got, name) if hasattr(got, name) else got[name]
        close(x, *want[name], steps, "grad_" + name)


BACKWARD = [(160, 1, 4096), (400, 3, 1024), (1000, 1, 200), (70, 130, 512), (40, 300, 1024),
            (400, 9, 264), (77, 5, 12288), (160, 1, 12288)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("per_batch", [False, True])
@pytest.mark.parametrize("B,S,D", BACKWARD)
def test_backward(rm, B, S, D, per_batch, dtype):
    t = Boundary(rm, B, S, D, dtype, per_batch)
    g = rm.sandwich_rmsnorm_modulate_backward(t.u, t.res, t.pw, t.gate, t.w, t.scale, t.gr, t.go,
                                              t.rp, t.r, residual_scale=0.5, update_scale=1.5)
    want = ref.sandwich_grad(t.u, t.res, t.pw, t.gate, t.w, t.scale, t.gr, t.go, t.stat(t.rp),
                             t.stat(t.r), 0.5, 1.5, t.rows, t.rows)
    close(g.residual, *want["residual"], chain.TERM, "grad_residual")
    close(g.update, *want["update"], chain.UPDATE, "grad_update")
    check_columns(t, g, want, ("post_weight", "gate", "weight", "scale", "shift"))


@pytest.mark.parametrize("per_batch", [False, True])
@pytest.mark.parametrize("B,S,D", BACKWARD)
def test_rms_backward(rm, B, S, D, per_batch):
    t = Boundary(rm, B, S, D, BF16, per_batch)
    gx, gw, gsc, gsh = rm.rmsnorm_modulate_backward(t.res, t.w, t.scale, t.go, t.r, grad_res=t.gr)
    want = {}
    dx, size = ref.norm_grad(t.res, t.w, t.scale, t.go, t.gr, t.stat(t.r), t.rows, want)
    close(gx, dx, size, chain.TERM, "grad_x")
    check_columns(t, dict(weight=gw, scale=gsc, shift=gsh), want, ("weight", "scale", "shift"))


def test_a_batch_does_not_depend_on_the_others(rm):
    for B, S, D in ((160, 3, 4096), (400, 2, 8200)):
        t = Boundary(rm, B, S, D, BF16, True)
        g = rm.sandwich_rmsnorm_modulate_backward(t.u, t.res, t.pw, t.gate, t.w, t.scale, t.gr,
                                                  t.go, t.rp, t.r)
        for b in (0, 75, B - 1):
            at, rows = slice(b, b + 1), slice(b * S, (b + 1) * S)
            res, out = rm.sandwich_rmsnorm_modulate(
                t.x[at], t.u[at], t.pw, t.gate[at], t.w, t.scale[at], t.shift[at],
                residual_scale=0.5, update_scale=1.5)
            assert torch.equal(res, t.res[at]) and torch.equal(out, t.out[at])
            h = rm.sandwich_rmsnorm_modulate_backward(
                t.u[at], t.res[at], t.pw, t.gate[at], t.w, t.scale[at], t.gr[at], t.go[at],
                t.rp[rows], t.r[rows])
            for name in ("residual", "update", "gate", "scale", "shift"):
                assert torch.equal(getattr(h, name), getattr(g, name)[at]), name
