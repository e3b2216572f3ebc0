"""The norms after and before a block and their gradients against the definition in float64.

Bounds, with u = 2^-24.  A stored value is off by at most its type's half step, eps / 2 of it.  The
fp32 evaluation before that: a row's sum adds at most 16 values in a thread, 5 steps in a warp and 32
warps' parts, so its relative error is under 53 u, half of that in 1 / sqrt; with the few products
around it every term is off by under 64 u of itself.  Where a mean enters a second time (grad_update)
the two errors add up: 128 u.  A column's sum adds at most 64 rows in an item, the items dealt to 8
warps, and the batches: under (64 + items / 8 + 8 + B + 64) u of the magnitudes summed."""
import pytest
import torch

import _sandwich as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


class Inputs:
    """Everything a block boundary has; the adaLN rows are strided views of one projection."""

    def __init__(self, B, S, D, dtype, per_batch=True, seed=0, gated=True, mod=True, weights=True):
        gen = torch.Generator(device="cuda").manual_seed(seed + 7 * D + S)
        n = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.B, self.S, self.D, self.dtype = B, S, D, dtype
        outlier = torch.where(torch.rand(B, S, 1, device="cuda", generator=gen) < 0.05, 20.0, 1.0)
        self.residual = (n(B, S, D) * outlier).to(dtype)
        self.update = (n(B, S, D) * outlier.flip(1)).to(dtype)
        self.rows = B if per_batch else 1
        cut = (0.3 * n(self.rows, 1, 3 * D)).to(dtype).chunk(3, -1)
        self.gate = cut[0] if gated else None
        self.scale, self.shift = (cut[1], cut[2]) if mod else (None, None)
        self.weight = (1 + 0.05 * n(D)).to(dtype) if weights else None
        self.post_weight = (1 + 0.05 * n(D)).to(dtype) if weights else None
        self.grad_out, self.grad_res = n(B, S, D).to(dtype), n(B, S, D).to(dtype)


def close(got, want, size, steps, what):
    f = torch.finfo(got.dtype)
    half = 0.0 if got.dtype == torch.float32 else f.eps / 2
    least = f.smallest_normal * f.eps
    bound = half * want.abs() + steps * U * size + least
    fine = want.abs() < float(f.max)
    off = ((got.double() - want).abs() / bound)[fine]
    assert got.isfinite()[fine].all(), what
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst} times its bound"


def forward(rm, t, residual_scale=1.0, update_scale=1.0, need_out=True, eps=1e-6, post_eps=None,
            **kw):
    n = t.B * t.S
    rp = torch.empty(n, dtype=torch.float32, device="cuda")
    r = torch.empty(n, dtype=torch.float32, device="cuda") if need_out else None
    res, out = rm.sandwich_rmsnorm_modulate(
        t.residual, t.update, t.post_weight, t.gate, t.weight, t.scale, t.shift, eps=eps,
        post_eps=post_eps, residual_scale=residual_scale, update_scale=update_scale,
        need_out=need_out, post_rstd_out=rp, rstd_out=r, **kw)
    return res, out, rp, r


def check_forward(rm, t, residual_scale=1.0, update_scale=1.0, need_out=True, eps=1e-6,
                  post_eps=None):
    before = t.residual.clone()
    res, out, rp, r = forward(rm, t, residual_scale, update_scale, need_out, eps, post_eps)
    pe = eps if post_eps is None else post_eps
    want, size = ref.residual_add(before, t.update, t.post_weight, t.gate, pe, residual_scale,
                                  update_scale)
    close(res, want, size, 64, "res")
    want = ref.rstd(t.update, pe).view(-1)
    close(rp, want, want, 64, "post_rstd")
    if need_out:
        want, size = ref.norm(res, t.weight, t.scale, t.shift, eps)
        close(out, want, size, 64, "out")
        want = ref.rstd(res, eps).view(-1)
        close(r, want, want, 64, "rstd")
    else:
        assert out is None
    return res, out, rp, r


SHAPES = [(1, 1, 8), (3, 5, 40), (2, 33, 256), (1, 77, 520), (2, 129, 1024), (4, 1, 4096),
          (1, 700, 4096), (2, 200, 3584), (1, 31, 6144), (2, 9, 8192), (1, 17, 8200),
          (2, 40, 12296), (1, 33, 16384)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,S,D", SHAPES)
def test_forward(rm, B, S, D, dtype):
    check_forward(rm, Inputs(B, S, D, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kw,call", [
    (dict(per_batch=False), dict(residual_scale=0.5, update_scale=1.5)),
    (dict(gated=False), dict(update_scale=0.25)),
    (dict(mod=False), dict(eps=1e-5, post_eps=1e-2)),
    (dict(weights=False), {}),
    (dict(gated=False, mod=False, weights=False), dict(residual_scale=-2.0)),
    ({}, dict(need_out=False)),
    (dict(gated=False, per_batch=False), dict(need_out=False, update_scale=0.0)),
])
def test_forward_parts(rm, kw, call, dtype):
    for B, S, D in ((2, 50, 1032), (2, 7, 256), (1, 9, 9216)):
        check_forward(rm, Inputs(B, S, D, dtype, **kw), **call)


def test_scale_or_shift_alone(rm):
    t = Inputs(2, 9, 512, torch.bfloat16)
    t.shift = None
    check_forward(rm, t)
    t = Inputs(2, 9, 512, torch.bfloat16)
    t.scale = None
    check_forward(rm, t)


def test_rows_do_not_depend_on_their_batch(rm):
    for D in (264, 4096, 10240):
        t = Inputs(3, 400, D, torch.bfloat16)
        res, out, rp, r = forward(rm, t)
        one = Inputs(3, 400, D, torch.bfloat16)
        for name in ("residual", "update"):
            setattr(one, name, getattr(one, name)[1:2, 5:6].contiguous())
        for name in ("gate", "scale", "shift"):
            setattr(one, name, getattr(one, name)[1:2])
        one.B, one.S = 1, 1
        a, b, _, _ = forward(rm, one)
        assert torch.equal(a, res[1:2, 5:6]) and torch.equal(b, out[1:2, 5:6])


def test_in_place_residual_and_given_outputs(rm):
    t = Inputs(2, 300, 2048, torch.bfloat16)
    res, out, _, _ = forward(rm, t)
    spare = torch.full_like(out, float("nan"))
    a, b, _, _ = forward(rm, t, res_out=t.residual, out=spare)
    assert a is t.residual and b is spare
    assert torch.equal(a, res) and torch.equal(b, out)


def test_rows_behind_the_last_stay(rm):
    t = Inputs(1, 5, 1024, torch.bfloat16)
    buf = torch.full((2, 8, 1024), 3.0, dtype=torch.bfloat16, device="cuda")
    forward(rm, t, res_out=buf[0, :5].unsqueeze(0), out=buf[1, :5].unsqueeze(0))
    assert (buf[:, 5:] == 3.0).all()


@pytest.mark.parametrize("D", [64, 4096, 9000])
def test_extreme_rows(rm, D):
    # rows whose squares leave fp32: huge, tiny (with a tiny eps), zero, one value alone
    t = Inputs(1, 8, D, torch.bfloat16, gated=False, mod=False, weights=False)
    gen = torch.Generator(device="cuda").manual_seed(D)
    base = torch.randn(8, D, device="cuda", generator=gen)
    size = torch.tensor([1e30, 1e-30, 0.0, 1e20, 1e-20, 1e36, 1e-36, 1.0], device="cuda")
    t.update = (base * size[:, None]).to(torch.bfloat16)[None].contiguous()
    t.update[0, 7] = 0.0
    t.update[0, 7, 3] = 3e38
    t.residual.zero_()
    for eps in (1e-6, 1e-30, 1e-38):
        check_forward(rm, t, eps=1e-6, post_eps=eps)
    # and the same rows through the norm after the add
    t.residual = t.update.clone()
    t.update = torch.zeros_like(t.update)
    for eps in (1e-6, 1e-30, 1e-38):
        check_forward(rm, t, eps=eps, post_eps=1e-6)


@pytest.mark.parametrize("B,S,D", [(1, 20000, 1024), (1, 9000, 4096), (2, 3100, 6144), (3, 700, 16384)])
def test_forward_long(rm, B, S, D):
    # many rows to a group of warps, whose rings are shorter by then
    check_forward(rm, Inputs(B, S, D, torch.bfloat16))


@pytest.mark.parametrize("D", [72, 4096, 12288])
def test_extreme_rows_in_turn(rm, D):
    # ordinary rows and those that take another way through the sums, next to one another in a group
    # of warps: every row's result is its own, whatever stands before and after it
    S = 4000
    gen = torch.Generator(device="cuda").manual_seed(D)
    size = torch.tensor([1.0, 0.0, 1e30, 1.0, 1e-30, float("inf"), 1e36, 0.0, 1.0, 1e-36, 1e20],
                        device="cuda")
    kind = size[torch.randint(0, len(size), (2, S, 1), device="cuda", generator=gen)]
    n = torch.randn(2, S, D, device="cuda", generator=gen)
    u, x = (n * kind).bfloat16()[:, None].unbind(0)
    flat = lambda t: t.view(torch.int32 if t.dtype is torch.float32 else torch.int16)  # noqa: E731

    def run(x, u):
        rp, r = (torch.empty(S, dtype=torch.float32, device="cuda") for _ in range(2))
        res, out = rm.sandwich_rmsnorm_modulate(x, u, eps=1e-30, post_eps=1e-38, post_rstd_out=rp,
                                                rstd_out=r)
        return res[0], out[0], rp, r

    there = run(x, u)
    order = torch.randperm(S, device="cuda", generator=gen)
    back = run(x[:, order].contiguous(), u[:, order].contiguous())
    for a, b in zip(there, back):
        a, b = a[order], b
        same = (flat(a) == flat(b)) | (a.isnan() & b.isnan())
        assert same.all()


def test_non_finite_rows_stay_alone(rm):
    t = Inputs(1, 6, 512, torch.bfloat16)
    res, out, _, _ = forward(rm, t)
    t.update[0, 2, 7] = float("nan")
    t.update[0, 4, 9] = float("inf")
    t.residual[0, 1, 3] = float("inf")
    a, b, _, _ = forward(rm, t)
    assert a[0, 2].isnan().all() and b[0, 2].isnan().all()
    # an infinite value: rstd 0, so NaN where it stands and the residual elsewhere
    assert a[0, 4, 9].isnan() and torch.equal(a[0, 4, 10:], t.residual[0, 4, 10:])
    assert a[0, 1, 3].isinf() and b[0, 1, 3].isnan()
    for row in (0, 3, 5):
        assert torch.equal(a[0, row], res[0, row]) and torch.equal(b[0, row], out[0, row])


def backward(rm, t, res, rp, r, residual_scale, update_scale, gr=True, go=True, **kw):
    return rm.sandwich_rmsnorm_modulate_backward(
        t.update, res, t.post_weight, t.gate, t.weight, t.scale, t.grad_res if gr else None,
        t.grad_out if go else None, rp, r, residual_scale=residual_scale,
        update_scale=update_scale, **kw)


def column_steps(t):
    return 64 + -(-t.S // 8) + 8 + t.B + 64


def check_backward(rm, t, residual_scale=1.0, update_scale=1.0, gr=True, go=True):
    res, _, rp, r = forward(rm, t, residual_scale, update_scale, need_out=go)
    g = backward(rm, t, res, rp, r, residual_scale, update_scale, gr, go)
    wide = lambda s: None if s is None else s.double().view(t.B, t.S, 1)  # noqa: E731
    want = ref.sandwich_grad(t.update, res, t.post_weight, t.gate, t.weight if go else None,
                             t.scale if go else None, t.grad_res if gr else None,
                             t.grad_out if go else None, wide(rp), wide(r), residual_scale,
                             update_scale, t.rows, t.rows)
    close(g.residual, *want["residual"], 64, "grad_residual")
    close(g.update, *want["update"], 128, "grad_update")
    for name, there in (("post_weight", t.post_weight), ("gate", t.gate),
                        ("weight", t.weight if go else None), ("scale", t.scale if go else None),
                        ("shift", t.scale if go else None)):
        x = getattr(g, name)
        if there is None:
            assert x is None
            continue
        assert x.dtype == torch.float32
        assert x.shape == ((t.D,) if "weight" in name else (t.rows, t.D))
        close(x, *want[name], column_steps(t), "grad_" + name)
    return g


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,S,D", SHAPES)
def test_backward(rm, B, S, D, dtype):
    check_backward(rm, Inputs(B, S, D, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kw,call", [
    (dict(per_batch=False), dict(residual_scale=0.5, update_scale=1.5)),
    (dict(gated=False), dict(update_scale=0.25)),
    (dict(mod=False), dict(gr=False)),
    (dict(weights=False), {}),
    (dict(gated=False, mod=False, weights=False), dict(residual_scale=-2.0)),
    ({}, dict(go=False)),
    (dict(per_batch=False), dict(go=False)),
])
def test_backward_parts(rm, kw, call, dtype):
    for B, S, D in ((2, 50, 1032), (3, 7, 256), (1, 9, 9216)):
        check_backward(rm, Inputs(B, S, D, dtype, **kw), **call)


def test_backward_long(rm):
    # more rows than one wave of items, of the largest chunks
    check_backward(rm, Inputs(2, 21000, 512, torch.bfloat16))
    check_backward(rm, Inputs(1, 10007, 1024, torch.float16, per_batch=False))


def test_backward_of_a_norm_against_differences(rm):
    # fp16 forward calls with steps large against the rounding: the slope of sum(out * go) along
    # one direction, central differences of three step sizes bracketing the analytic value
    t = Inputs(1, 4, 512, torch.bfloat16)
    res, _, rp, r = forward(rm, t)
    g = backward(rm, t, res, rp, r, 1.0, 1.0)
    gen = torch.Generator(device="cuda").manual_seed(5)
    way = torch.randn(t.update.shape, device="cuda", generator=gen).double()

    def loss(step):
        u = t.update.double() + step * way
        h, _ = ref.residual_add(t.residual, u, t.post_weight, t.gate, 1e-6, 1.0, 1.0)
        o, _ = ref.norm(h, t.weight, t.scale, t.shift, 1e-6)
        return ((h * t.grad_res.double()).sum() + (o * t.grad_out.double()).sum()).item()

    slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
    # the gradient's rounding (eps / 2 of each term) and that of res, which the call is given rounded
    size = (g.update.double() * way).abs().sum().item()
    assert abs((g.update.double() * way).sum().item() - slope) <= 2 * 2.0 ** -8 * size


def test_backward_is_batch_invariant_and_repeatable(rm):
    for D in (512, 4096):
        t = Inputs(3, 500, D, torch.bfloat16)
        res, _, rp, r = forward(rm, t)
        a, b = (backward(rm, t, res, rp, r, 1.0, 1.0) for _ in range(2))
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        one = rm.sandwich_rmsnorm_modulate_backward(
            t.update[1:2], res[1:2], t.post_weight, t.gate[1:2], t.weight, t.scale[1:2],
            t.grad_res[1:2], t.grad_out[1:2], rp[500:1000], r[500:1000])
        for name in ("residual", "update", "gate", "scale", "shift"):
            assert torch.equal(getattr(one, name)[0], getattr(a, name)[1]), name


def test_backward_selects(rm):
    t = Inputs(2, 40, 512, torch.bfloat16)
    res, _, rp, r = forward(rm, t)
    a = backward(rm, t, res, rp, r, 1.0, 1.0)
    x = backward(rm, t, res, rp, r, 1.0, 1.0, need_mod=False)
    m = backward(rm, t, res, rp, r, 1.0, 1.0, need_x=False)
    assert torch.equal(x.residual, a.residual) and torch.equal(x.update, a.update)
    assert x.gate is None and x.weight is None and x.shift is None
    assert m.residual is None and m.update is None
    for name in ("post_weight", "gate", "weight", "scale", "shift"):
        assert torch.equal(getattr(m, name), getattr(a, name)), name
    need = rm.library().sandwich_rmsnorm_modulate_backward_workspace_bytes(2, 40, 512)
    # stale bytes in the workspace do not matter
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    w = backward(rm, t, res, rp, r, 1.0, 1.0, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(a, w))


def test_expanded_row_gets_one_gradient(rm):
    t = Inputs(3, 20, 256, torch.bfloat16, per_batch=False)
    res, _, rp, r = forward(rm, t)
    a = backward(rm, t, res, rp, r, 1.0, 1.0)
    t.gate, t.scale = t.gate.expand(3, 1, 256), t.scale.expand(3, 1, 256)
    b = backward(rm, t, res, rp, r, 1.0, 1.0)
    assert a.gate.shape == b.gate.shape == (1, 256)
    assert torch.equal(a.gate, b.gate) and torch.equal(a.scale, b.scale)


def test_shapes_of_rows(rm):
    # [S, D] tensors, and row vectors as [D], [1, D] and [B, D]: the same bits as [B, S, D] with
    # [B, 1, D]
    def both(t, two=lambda x: x, rows=lambda x: x):
        r, rp = (torch.empty(t.B * t.S, dtype=torch.float32, device="cuda") for _ in range(2))
        g, sc, sh = rows(t.gate), rows(t.scale), rows(t.shift)
        u = two(t.update)
        res, out = rm.sandwich_rmsnorm_modulate(two(t.residual), u, t.post_weight, g, t.weight, sc,
                                                sh, post_rstd_out=rp, rstd_out=r)
        grads = rm.sandwich_rmsnorm_modulate_backward(u, res, t.post_weight, g, t.weight, sc,
                                                      two(t.grad_res), two(t.grad_out), rp, r)
        return [res, out, *grads]

    one, three = Inputs(1, 37, 520, torch.bfloat16), Inputs(3, 37, 520, torch.bfloat16)
    for t, two, rows in ((one, lambda x: x[0], lambda x: x[0]), (one, lambda x: x[0], lambda x: x[0, 0]),
                         (one, lambda x: x, lambda x: x[0, 0]), (three, lambda x: x, lambda x: x[:, 0])):
        for a, b in zip(both(t), both(t, two, rows)):
            assert torch.equal(a.reshape(-1), b.reshape(-1))


def test_statistics_are_any_shape(rm):
    t = Inputs(2, 5, 128, torch.float16)
    a, b = (torch.empty(2, 5, 1, dtype=torch.float32, device="cuda") for _ in range(2))
    rm.sandwich_rmsnorm_modulate(t.residual, t.update, post_rstd_out=a, rstd_out=b)
    want = ref.rstd(t.update, 1e-6)
    close(a, want, want, 64, "post_rstd")


def check_rms(rm, t, gr=True):
    rstd = torch.empty(t.B * t.S, dtype=torch.float32, device="cuda")
    rm.rmsnorm_modulate(t.residual, t.weight, t.scale if t.scale is not None else
                        torch.zeros(t.D, dtype=t.dtype, device="cuda"),
                        t.shift if t.shift is not None else
                        torch.zeros(t.D, dtype=t.dtype, device="cuda"), rstd_out=rstd)
    gx, gw, gsc, gsh = rm.rmsnorm_modulate_backward(t.residual, t.weight, t.scale, t.grad_out, rstd,
                                                    grad_res=t.grad_res if gr else None)
    want = {}
    dx, size = ref.norm_grad(t.residual, t.weight, t.scale, t.grad_out, t.grad_res if gr else None,
                             rstd.double().view(t.B, t.S, 1), t.rows, want)
    close(gx, dx, size, 64, "grad_x")
    for name, x, there in (("weight", gw, t.weight), ("scale", gsc, t.scale),
                           ("shift", gsh, t.scale)):
        if there is None:
            assert x is None
        else:
            close(x, *want[name], column_steps(t), "grad_" + name)


@pytest.mark.parametrize("B,S,D", SHAPES)
def test_rms_backward(rm, B, S, D):
    check_rms(rm, Inputs(B, S, D, torch.bfloat16), gr=S % 2 == 0)


@pytest.mark.parametrize("kw", [dict(per_batch=False), dict(mod=False), dict(weights=False),
                                dict(mod=False, weights=False)])
def test_rms_backward_parts(rm, kw):
    for B, S, D in ((2, 50, 1032), (3, 8, 256), (1, 10, 9216)):
        for gr in (False, True):
            check_rms(rm, Inputs(B, S, D, torch.bfloat16, **kw), gr)


def test_no_tokens(rm):
    t = Inputs(2, 0, 256, torch.bfloat16)
    res, out, rp, r = forward(rm, t)
    assert res.shape == out.shape == (2, 0, 256)
    g = backward(rm, t, res, rp, r, 1.0, 1.0)
    for x in (g.post_weight, g.gate, g.weight, g.scale, g.shift):
        assert (x == 0).all()
    assert g.gate.shape == (2, 256)
    _, gw, gsc, gsh = rm.rmsnorm_modulate_backward(t.residual, t.weight, t.scale, t.grad_out, r)
    assert (gw == 0).all() and (gsc == 0).all() and (gsh == 0).all()


def test_streams_and_graphs(rm):
    t = Inputs(2, 300, 1024, torch.bfloat16)
    res, out, rp, r = forward(rm, t)
    want = backward(rm, t, res, rp, r, 1.0, 1.0)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [(forward(rm, t, stream=s)[0], backward(rm, t, res, rp, r, 1.0, 1.0, stream=s))
           for _ in range(8) for s in streams]
    torch.cuda.synchronize()
    for a, g in got:
        assert torch.equal(a, res) and all(torch.equal(x, y) for x, y in zip(g, want))
    # two captured steps on other data, replayed in turn
    graphs = []
    for seed in (1, 2):
        q = Inputs(2, 300, 1024, torch.bfloat16, seed=seed)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            a, b, p, s = forward(rm, q)
            g = backward(rm, q, a, p, s, 1.0, 1.0)
        graphs.append((graph, q, a, b, p, s, g))
    for _ in range(3):
        for item in graphs:
            item[0].replay()
    torch.cuda.synchronize()
    for _, q, a, b, p, s, g in graphs:
        a2, b2, p2, s2 = forward(rm, q)
        g2 = backward(rm, q, a2, p2, s2, 1.0, 1.0)
        assert torch.equal(a, a2) and torch.equal(b, b2)
        assert all(torch.equal(x, y) for x, y in zip(g, g2))


def test_gpu_refusals(rm):
    t = Inputs(2, 6, 64, torch.bfloat16)
    call = lambda **k: rm.sandwich_rmsnorm_modulate(  # noqa: E731
        k.get("x", t.residual), k.get("u", t.update), k.get("pw"), k.get("g"), k.get("w"),
        k.get("sc"), k.get("sh"), **{n: v for n, v in k.items() if len(n) > 2})
    half = torch.zeros(2, 6, 64, dtype=torch.float16, device="cuda")
    for k in (dict(u=half), dict(pw=half[0, 0]), dict(g=half[:, :1])):
        with pytest.raises(TypeError):
            call(**k)
    for k in (dict(u=t.update[:1]), dict(pw=t.update[0, 0, :8]), dict(g=t.update[:, :2]),
              dict(x=t.residual.transpose(0, 1)), dict(need_out=False, out=t.grad_out),
              dict(sc=t.update[:, :1], sh=t.update[:1, :1]),
              dict(post_rstd_out=torch.empty(3, device="cuda")),
              dict(w=torch.ones(64, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            call(**k)
    with pytest.raises(rm.RmsmodError):  # out over the residual
        call(out=t.residual)
    res, _, rp, r = forward(rm, t)
    with pytest.raises(ValueError):
        backward(rm, t, res, rp, r, 1.0, 1.0, gr=False, go=False)
    with pytest.raises(ValueError):
        backward(rm, t, res, None, r, 1.0, 1.0)
    with pytest.raises(ValueError):
        backward(rm, t, res, rp, None, 1.0, 1.0)
    with pytest.raises(ValueError):
        backward(rm, t, res, rp, r, 1.0, 1.0,
                 workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
