"""The norm before an 8-bit projection and the gradients that 8-bit checkpoints give, against their
definitions in 64 bits.

Bounds: res is one rounding of a sum that fp32 holds to 2^-24.  rstd is good to D / 32 + 16 roundings of
2^-24 of the squares' sum (whose order keeps fewer, all of one sign's), halved by the root, and three
more; each stored value has it, its products' 2^-24 and its own half step.  Column sums of n terms:
n * 2^-24 of the magnitudes summed, the bound of any order."""
import numpy as np
import pytest
import torch

import _mx8

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
EPS = 1e-6


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


def ulps(D):
    return (D / 64 + 12) * 2.0 ** -24


class Case:
    def __init__(self, B, S, D, dtype, per_batch=True, mod=True, weight=True, shift=None, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed + B * S + D)
        n = lambda *s, std=1.0, mean=0.0: (  # noqa: E731
            torch.randn(*s, device="cuda", generator=gen) * std + mean).to(dtype)
        self.B, self.S, self.D, self.dtype, self.per_batch = B, S, D, dtype, per_batch
        size = torch.exp2(torch.randint(-4, 5, (B, S, 1), device="cuda", generator=gen).float())
        self.x, self.update = n(B, S, D) * size.to(dtype), n(B, S, D)
        self.weight = n(D, std=0.1, mean=1.0) if weight else None
        cut = n(B if per_batch else 1, 1, 3 * D, std=0.3).chunk(3, -1)
        self.scale = cut[1] if mod else None
        self.shift = cut[2] if (mod if shift is None else shift) else None
        self.go, self.gr = n(B, S, D), n(B, S, D)

    def m64(self):
        one = torch.ones(1, 1, self.D, dtype=torch.float64, device="cuda")
        w = one if self.weight is None else self.weight.double() * one
        s = one if self.scale is None else 1.0 + self.scale.double()
        t = 0.0 * one if self.shift is None else self.shift.double()
        return w, s, t


def check_norm(rm, c, update=True, keep=True, eps=EPS, res_out=None):
    rstd = torch.empty(c.B * c.S, device="cuda")
    x = c.x.clone()
    want = x.double() + (c.update.double() if update else 0.0)
    res, out, kept = rm.add_rmsnorm_mxfp8(x, c.update if update else None, c.weight, c.scale, c.shift,
                                          eps=eps, keep=keep, rstd_out=rstd,
                                          res_out=x if res_out == "x" else None)
    if update:
        off = (res.double() - want).abs()
        assert (off <= _mx8.step_of(want, c.dtype) + 2.0 ** -24 * want.abs()).all()
    else:
        assert res is x and torch.equal(x, c.x)
    h = res.double()
    r = (h.square().mean(-1) + eps).rsqrt()
    # (a root past fp32's range is its Inf, which the rows' results do not go through)
    past, got = r > float(torch.finfo(torch.float32).max), rstd.double().view(c.B, c.S)
    assert torch.isinf(got[past]).all()
    assert ((got - r).abs() <= ulps(c.D) * r)[~past].all()
    w, s, t = c.m64()
    y = h * r[..., None] * w * s
    slack = (ulps(c.D) + 6 * 2.0 ** -24) * y.abs() + 2.0 ** -24 * (y + t).abs()
    _mx8.check_held(out, y + t, slack)
    if keep:
        codes, e = _mx8.quantize(res.reshape(-1, c.D).double().cpu().numpy())
        got, _, flat = _mx8.shown(kept)
        assert np.array_equal(got, codes) and np.array_equal(flat, _mx8.tiles(e, c.D))
    else:
        assert kept is None
    return res, out, kept, rstd


SHAPES = [(1, 1, 32), (1, 3, 64), (2, 77, 160), (1, 128, 256), (3, 43, 512), (1, 129, 544),
          (2, 65, 1024), (1, 100, 2080), (4, 1, 4096), (2, 33, 4128), (1, 40, 6144), (1, 9, 8192),
          (1, 7, 8224), (2, 18, 16384)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,S,D", SHAPES)
def test_norm(rm, B, S, D, dtype):
    check_norm(rm, Case(B, S, D, dtype))


@pytest.mark.parametrize("update,keep,per_batch,mod,weight,shift", [
    (False, False, False, True, True, None), (True, False, True, False, True, None),
    (False, True, False, False, False, None), (True, True, True, False, True, True),
    (True, True, False, True, False, False),
])
def test_norm_parts(rm, update, keep, per_batch, mod, weight, shift):
    check_norm(rm, Case(3, 50, 672, torch.bfloat16, per_batch, mod, weight, shift), update, keep)


def test_norm_in_place_and_other_forms(rm):
    c = Case(2, 70, 1056, torch.float16)
    res, out, kept, rstd = check_norm(rm, c, res_out="x")
    # [S, D] tensors, outputs given, the update's place taken
    u = c.update[0].clone()
    o, k = (rm.mxfp8_quantize(torch.ones_like(u)) for _ in range(2))
    row = lambda t: t[0, 0].contiguous()  # noqa: E731
    got = rm.add_rmsnorm_mxfp8(c.x[0].contiguous(), u, c.weight, row(c.scale), row(c.shift), keep=k,
                               out=o, res_out=u)
    assert got[0] is u and got[1] is o and got[2] is k
    assert torch.equal(u, res[0])
    same = lambda a, b: torch.equal(a.codes.view(torch.uint8), b.codes[0].view(torch.uint8))  # noqa
    assert same(o, out) and same(k, kept)


def test_norm_rows_do_not_depend_on_their_place(rm):
    c = Case(1, 300, 992, torch.bfloat16, per_batch=False)
    _, out, kept, rstd = check_norm(rm, c)
    part = torch.empty(45, device="cuda")
    _, o, k = rm.add_rmsnorm_mxfp8(c.x[0, 201:246], c.update[0, 201:246], c.weight, c.scale, c.shift,
                                   keep=True, rstd_out=part)
    assert torch.equal(part, rstd[201:246])
    for a, b in ((o, out), (k, kept)):
        ca, ga, _ = _mx8.shown(a)
        cb, gb, _ = _mx8.shown(b)
        assert np.array_equal(ca, cb[201:246]) and np.array_equal(ga, gb[201:246])


@pytest.mark.parametrize("D", [64, 4096, 16384])
def test_norm_of_extreme_rows(rm, D):
    # squares past fp32, or under it: the statistics are those of the values all the same
    x = torch.randn(9, D, device="cuda").bfloat16()
    size = torch.tensor([1e30, 3e37, 1e25, 1.0, 1e-25, 1e-37, 1e-40, 0.0, 1e19], device="cuda")
    c = Case(1, 9, D, torch.bfloat16, mod=False)
    c.x = (x.double() * size[:, None].double()).bfloat16().view(1, 9, D)
    for eps in (EPS, 1e-30, 0.0):
        if eps == 0.0:
            c.x[0, 7] = 1e-39  # no row of zeros without eps
        check_norm(rm, c, update=False, eps=eps)


def test_norm_of_rows_that_are_not_finite(rm):
    c = Case(1, 6, 128, torch.bfloat16)
    c.x[0, 1, 5], c.x[0, 2, 7], c.x[0, 3, 9] = float("inf"), float("nan"), -float("inf")
    rstd = torch.empty(6, device="cuda")
    _, out, kept = rm.add_rmsnorm_mxfp8(c.x, None, c.weight, c.scale, c.shift, keep=True,
                                        rstd_out=rstd)
    bad, k = torch.isnan(rm.mxfp8_dequantize(out)[0]), torch.isnan(rm.mxfp8_dequantize(kept)[0])
    assert rstd[1] == 0 and torch.isnan(rstd[2]) and rstd[3] == 0
    assert not bad[[0, 4, 5]].any() and not k[[0, 4, 5]].any()
    # Inf * 0 in its block; the others are the shift alone
    assert bad[1, :32].all() and not bad[1, 32:].any() and bad[2].all() and bad[3, :32].all()
    assert k[1, :32].all() and not k[1, 32:].any() and k[2, :32].all() and not k[2, 32:].any()


def test_norm_leaves_what_lies_behind_its_rows(rm):
    c = Case(1, 37, 96, torch.bfloat16, per_batch=False)
    codes = torch.full((40, 96), 3.0, device="cuda").to(torch.float8_e4m3fn)
    buf = torch.full((40, 96), 5.0, dtype=torch.bfloat16, device="cuda")
    out = rm.Mxfp8(codes[:37], torch.full((512,), 9, dtype=torch.uint8, device="cuda"))
    rm.add_rmsnorm_mxfp8(c.x[0], c.update[0], c.weight, c.scale, c.shift, out=out, res_out=buf[:37])
    assert (codes[37:].float() == 3.0).all() and (buf[37:] == 5.0).all()
    _, g, flat = _mx8.shown(out)
    assert np.array_equal(flat, _mx8.tiles(g, 96))


# ---------------------------------------------------------------------------------------------
# the norm's gradients
# ---------------------------------------------------------------------------------------------

def norm_grads64(c, h, r, gr):
    w, s, _ = c.m64()
    r = r.double().view(c.B, c.S, 1)
    hh = h * r
    go = c.go.double()
    d = go * w * s
    dx = r * (d - hh * (d * hh).mean(-1, keepdim=True))
    size = r * (d.abs() + hh.abs() * (d * hh).abs().mean(-1, keepdim=True))
    if gr is not None:
        dx = dx + gr.double()
        size = size + gr.double().abs()
    fold = (lambda t: t.sum(1)) if c.per_batch else (lambda t: t.sum((0, 1))[None])  # noqa: E731
    p = go * hh
    sums = {"weight": (p * s).sum((0, 1)), "scale": fold(p) * w[0], "shift": fold(go)}
    mags = {"weight": (p * s).abs().sum((0, 1)), "scale": fold(p.abs()) * w[0].abs(),
            "shift": fold(go.abs())}
    return dx, size, sums, mags


def check_norm_grad(rm, c, stream=True, **kw):
    codes, e = _mx8.quantize(c.x.reshape(-1, c.D).double().cpu().numpy())
    kept = _mx8.held(rm, codes, e)
    kept = rm.Mxfp8(kept.codes.view(c.B, c.S, c.D), kept.scales)
    h = _mx8.decoded(kept)
    rstd = (c.x.double().square().mean(-1) + EPS).rsqrt().float().view(-1)
    gr = c.gr if stream else None
    dx, size, sums, mags = norm_grads64(c, h, rstd, gr)
    got = rm.rmsnorm_mxfp8_backward(kept, c.weight, c.scale, c.go, rstd, grad_res=gr,
                                    shift=c.shift, **kw)
    if kw.get("need_x", True):
        bound = _mx8.step_of(dx, c.dtype) * (1 + 2.0 ** -10) + (c.D / 32 + 16) * 2.0 ** -24 * size
        assert got[0].dtype == c.dtype and ((got[0].double() - dx).abs() <= bound).all()
    else:
        assert got[0] is None
    wanted = {"weight": c.weight is not None, "scale": c.scale is not None,
              "shift": c.scale is not None or c.shift is not None}
    for (name, need), g in zip(wanted.items(), got[1:]):
        if not (need and kw.get("need_mod", True)):
            assert g is None
            continue
        n = c.B * c.S + 8
        assert g.dtype == torch.float32 and g.shape == sums[name].shape
        assert ((g.double() - sums[name]).abs() <= n * 2.0 ** -24 * mags[name] + 1e-30).all(), name
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,S,D", [(1, 1, 32), (1, 5, 64), (2, 77, 160), (3, 43, 512), (1, 300, 544),
                                   (2, 65, 1024), (1, 700, 2080), (4, 1, 4096), (2, 170, 4096),
                                   (2, 33, 4128), (1, 400, 6144), (1, 20, 8192), (3, 7, 8224),
                                   (2, 90, 16384)])
def test_norm_grad(rm, B, S, D, dtype):
    check_norm_grad(rm, Case(B, S, D, dtype))


@pytest.mark.parametrize("stream,per_batch,mod,weight,shift,kw", [
    (False, False, True, True, None, {}), (True, True, False, True, None, {}),
    (False, True, False, False, True, {}), (True, False, True, False, False, {}),
    (True, True, True, True, None, dict(need_x=False)),
    (False, False, True, True, None, dict(need_mod=False)),
    (True, True, False, False, None, {}),
])
def test_norm_grad_parts(rm, stream, per_batch, mod, weight, shift, kw):
    check_norm_grad(rm, Case(3, 90, 672, torch.bfloat16, per_batch, mod, weight, shift), stream, **kw)


def test_norm_grad_of_many_batches(rm):
    for B, S in ((700, 3), (5000, 1)):
        for per_batch in (True, False):
            check_norm_grad(rm, Case(B, S, 256, torch.bfloat16, per_batch))


def test_norm_grad_batches_do_not_depend_on_one_another(rm):
    c = Case(3, 130, 736, torch.bfloat16)
    gx, _, gs, gh = check_norm_grad(rm, c)
    one = Case(1, 130, 736, torch.bfloat16)
    for name in ("x", "go", "gr", "scale", "shift"):
        setattr(one, name, getattr(c, name)[1:2])
    one.weight = c.weight
    ox, _, os, oh = check_norm_grad(rm, one)
    # (a row of its own is every batch's: the same runs)
    assert torch.equal(ox[0], gx[1]) and torch.equal(os[0], gs[1]) and torch.equal(oh[0], gh[1])


def test_norm_grad_against_differences(rm):
    # the formula itself: finite differences of the norm in 64 bits at the checkpoint's values
    c = Case(1, 2, 64, torch.bfloat16)
    codes, e = _mx8.quantize(c.x.reshape(-1, 64).double().cpu().numpy())
    h = torch.from_numpy(_mx8.values(codes, e)).view(1, 2, 64).cuda()
    w, s, t = c.m64()
    f = lambda h: ((h * (h.square().mean(-1, keepdim=True) + EPS).rsqrt() * w * s + t)  # noqa: E731
                   * c.go.double()).sum((0, 2))
    rstd = (h.square().mean(-1) + EPS).rsqrt()
    dx = norm_grads64(c, h, rstd, None)[0]
    for i in (0, 7, 40, 63):
        step = torch.zeros_like(h)
        step[..., i] = 1e-5
        diff = (f(h + step) - f(h - step)) / 2e-5
        assert torch.allclose(diff, dx[0, :, i], rtol=1e-6, atol=1e-8)


# ---------------------------------------------------------------------------------------------
# the activation's gradient
# ---------------------------------------------------------------------------------------------

def check_act_grad(rm, B, S, N, dtype, act, gate=None, seed=0, need_sums=True):
    rng = np.random.default_rng(seed + B * S + N)
    codes, e = _mx8.quantize(rng.standard_normal((B * S, N)) * np.exp2(rng.integers(-3, 3, (B * S, 1))))
    held = _mx8.held(rm, codes, e)
    z = rm.Mxfp8(held.codes.view(B, S, N), held.scales)
    half = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(dtype).cuda()  # noqa: E731
    g = half(B, S, N)
    gt = half(B if gate == "batch" else 1, 1, 3 * N).chunk(3, -1)[2] if gate else None
    v = _mx8.decoded(z)
    h, slope = _mx8.activation(act, v)
    gv = torch.ones(1, 1, N, device="cuda", dtype=torch.float64) if gt is None else gt.double()
    dz = g.double() * slope * gv
    # near its zero the derivative is a difference of terms of up to 1
    slack = 2.0 ** -20 * (g.double() * gv).abs() * (1 if act else 0) + 2.0 ** -22 * dz.abs()
    grad_z, grad_bias, grad_gate = rm.mxfp8_activation_backward(z, g, activation=act, gate=gt,
                                                                need_sums=need_sums)
    assert grad_z.codes.shape == (B, S, N)
    _mx8.check_held(grad_z, dz, slack)
    if not need_sums:
        assert grad_bias is None and grad_gate is None
        return grad_z, None, None
    n = B * S + 8
    bound = n * 2.0 ** -24 * dz.abs().sum((0, 1)) + slack.sum((0, 1)) + 1e-30
    assert ((grad_bias.double() - dz.sum((0, 1))).abs() <= bound).all()
    if gate:
        t = g.double() * h
        fold = (lambda t: t.sum(1)) if gate == "batch" else (lambda t: t.sum((0, 1))[None])  # noqa
        bound = (n * 2.0 ** -24 + 2.0 ** -18) * fold(t.abs()) + 1e-30
        assert grad_gate.shape == (B if gate == "batch" else 1, N)
        assert ((grad_gate.double() - fold(t)).abs() <= bound).all()
    else:
        assert grad_gate is None
    return grad_z, grad_bias, grad_gate


@pytest.mark.parametrize("act", _mx8.ACTIVATIONS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,S,N,gate", [
    (1, 1, 32, None), (2, 77, 96, "batch"), (1, 128, 160, "one"), (3, 100, 416, "batch"),
    (1, 300, 1024, None), (2, 256, 128, "batch"), (5, 27, 4096, "batch"), (2, 200, 64, "one"),
])
def test_act_grad(rm, B, S, N, gate, dtype, act):
    check_act_grad(rm, B, S, N, dtype, act, gate)


def test_act_grad_without_sums(rm):
    check_act_grad(rm, 2, 150, 224, torch.bfloat16, "silu", "batch", need_sums=False)


def test_act_grad_of_many_batches(rm):
    check_act_grad(rm, 3000, 1, 64, torch.bfloat16, "gelu", "batch")
    check_act_grad(rm, 70000, 1, 32, torch.bfloat16, None, "batch")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_act_grad_at_far_arguments(rm, act):
    # every magnitude a block can have: neither end overflows on the way
    z = torch.zeros(2, 128, 64, dtype=torch.bfloat16, device="cuda")
    size = 2.0 ** torch.arange(-100, 28, device="cuda").double().view(128, 1)
    z[0], z[1] = size.bfloat16(), -size.bfloat16()
    q = rm.mxfp8_quantize(z)
    g = torch.ones_like(z)
    h, slope = _mx8.activation(act, _mx8.decoded(q))
    grad_z, _, grad_gate = rm.mxfp8_activation_backward(q, g, activation=act, gate=g[:, :1])
    _mx8.check_held(grad_z, slope, 2.0 ** -20 + 0 * slope)
    assert torch.isfinite(grad_gate).all()
    big = torch.full((1, 64), 3e38, dtype=torch.bfloat16, device="cuda")
    for s, want in ((1, 1.0), (-1, 0.0)):
        t, _, _ = rm.mxfp8_activation_backward(rm.mxfp8_quantize(s * big), g[0, :1], activation=act)
        assert (rm.mxfp8_dequantize(t) == want).all()


def test_act_grad_batches_do_not_depend_on_one_another(rm):
    rng = np.random.default_rng(3)
    z = torch.from_numpy(rng.standard_normal((3, 150, 96))).bfloat16().cuda()
    g = torch.from_numpy(rng.standard_normal((3, 150, 96))).bfloat16().cuda()
    gate = torch.from_numpy(rng.standard_normal((3, 1, 96))).bfloat16().cuda()
    _, _, whole = rm.mxfp8_activation_backward(rm.mxfp8_quantize(z), g, "silu", gate)
    _, _, two = rm.mxfp8_activation_backward(rm.mxfp8_quantize(z[1:].contiguous()), g[1:], "silu",
                                             gate[1:])
    assert torch.equal(whole[1:], two)


def test_act_grad_nan_stays_in_its_block(rm):
    z = torch.randn(3, 96, device="cuda").bfloat16()
    z[1, 40] = float("nan")
    t, _, _ = rm.mxfp8_activation_backward(rm.mxfp8_quantize(z), torch.ones_like(z), "gelu_tanh")
    bad = torch.isnan(rm.mxfp8_dequantize(t))
    assert bad[1, 32:64].all() and bad.sum() == 32


@pytest.mark.parametrize("act", _mx8.ACTIVATIONS)
@pytest.mark.parametrize("rows,N,lo,hi", [
    (130, 96, 108, 134),    # both sides of the scales whose derivatives are looked up
    (37, 64, 0, 40), (37, 64, 160, 200),
    (2500, 4128, 111, 131),  # more pieces than run at a time
])
def test_act_grad_under_every_scale(rm, rows, N, lo, hi, act):
    codes, e = _mx8.random_codes(np.random.default_rng(rows + lo), rows, N, lo, hi)
    z = _mx8.held(rm, codes, e)
    g = torch.from_numpy(np.random.default_rng(1).standard_normal((rows, N))).bfloat16().cuda()
    h, slope = _mx8.activation(act, _mx8.decoded(z))
    dz = g.double() * slope
    grad_z, grad_bias, _ = rm.mxfp8_activation_backward(z, g, activation=act)
    slack = 2.0 ** -20 * g.double().abs() * (1 if act else 0) + 2.0 ** -22 * dz.abs()
    _mx8.check_held(grad_z, dz, slack)
    bound = (rows + 8) * 2.0 ** -24 * dz.abs().sum(0) + slack.sum(0) + 1e-30
    assert ((grad_bias.double() - dz.sum(0)).abs() <= bound).all()


@pytest.mark.parametrize("act", _mx8.ACTIVATIONS)
def test_gate_grad_of_large_values(rm, act):
    # powers of two that the activation leaves as they are or takes to zero: the sum is exact
    z = torch.zeros(1, 3, 64, dtype=torch.bfloat16, device="cuda")
    z[0, 0], z[0, 1, :32], z[0, 2, :32] = 2.0 ** 44, 2.0 ** 100, -2.0 ** 90
    g = torch.full_like(z, 0.5)
    _, _, grad_gate = rm.mxfp8_activation_backward(rm.mxfp8_quantize(z), g, act, g[:, :1])
    want = torch.full((64,), 2.0 ** 43, dtype=torch.float64, device="cuda")
    want[:32] += 2.0 ** 99 - (2.0 ** 89 if act is None else 0.0)
    assert torch.equal(grad_gate[0], want.float())


@pytest.mark.parametrize("D", [256, 288, 4096, 4128, 5120, 5152, 6144, 6176, 8192, 8224, 16352])
def test_norm_either_side_of_its_variants(rm, D):
    # the widths at which a row goes to more vectors a thread, or to fewer groups
    c = Case(2, 40, D, torch.bfloat16)
    check_norm(rm, c)
    check_norm_grad(rm, c)
