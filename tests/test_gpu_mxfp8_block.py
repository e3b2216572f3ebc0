"""The 8-bit operators as a training step of a feed-forward block runs them -- the norm, two
projections, and all gradients from the checkpoints -- each result against its definition in 64 bits
of what the step gave the call; the same step on another stream, captured and replayed, and with what
the calls refuse."""
import numpy as np
import pytest
import torch

import _mx8

pytestmark = pytest.mark.gpu

B, S, D, F = 2, 83, 160, 416
EPS = 1e-6


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


def inputs(rm, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n = lambda *s, std=1.0: (torch.randn(*s, device="cuda", generator=gen) * std).bfloat16()  # noqa
    t = dict(x=n(B, S, D), update=n(B, S, D), weight=n(D, std=0.1) + 1.0, b1=n(F, std=0.1),
             b2=n(D, std=0.1), gy=n(B, S, D))
    t["scale"], t["shift"], t["gate"] = n(B, 1, 3 * D, std=0.3).chunk(3, -1)
    t["w1"], t["w2"] = n(F, D, std=D ** -0.5), n(D, F, std=F ** -0.5)
    return t


def step(rm, t, stream=None):
    k = dict(stream=stream)
    w1, w2 = rm.mxfp8_quantize(t["w1"], **k), rm.mxfp8_quantize(t["w2"], **k)
    res, h, kept = rm.add_rmsnorm_mxfp8(t["x"], t["update"], t["weight"], t["scale"], t["shift"],
                                        eps=EPS, keep=True, **k)
    rstd = torch.empty(B * S, device="cuda")
    # (the statistics of a second call: the same bits)
    rm.add_rmsnorm_mxfp8(t["x"], t["update"], t["weight"], t["scale"], t["shift"], eps=EPS,
                         rstd_out=rstd, **k)
    a, z1 = rm.mxfp8_linear(h, w1, bias=t["b1"], activation="gelu_tanh", quantize=True, keep=True, **k)
    y, z2 = rm.mxfp8_linear(a, w2, bias=t["b2"], gate=t["gate"], residual=res, keep=True, **k)
    dz2, db2, dgate = rm.mxfp8_activation_backward(z2, t["gy"], gate=t["gate"], **k)
    da = rm.mxfp8_linear(dz2, rm.mxfp8_transpose(w2, **k), **k)
    dw2 = rm.mxfp8_linear(rm.mxfp8_transpose(dz2, **k), rm.mxfp8_transpose(a, **k),
                          dtype=torch.float32, **k)
    dz1, db1, _ = rm.mxfp8_activation_backward(z1, da, "gelu_tanh", **k)
    dh = rm.mxfp8_linear(dz1, rm.mxfp8_transpose(w1, **k), **k)
    dw1 = rm.mxfp8_linear(rm.mxfp8_transpose(dz1, **k), rm.mxfp8_transpose(h, **k),
                          dtype=torch.float32, **k)
    dx, dw, dscale, dshift = rm.rmsnorm_mxfp8_backward(kept, t["weight"], t["scale"], dh, rstd,
                                                       grad_res=t["gy"], **k)
    return dict(w1=w1, w2=w2, res=res, h=h, kept=kept, rstd=rstd, a=a, z1=z1, y=y, z2=z2, dz2=dz2,
                db2=db2, dgate=dgate, da=da, dw2=dw2, dz1=dz1, db1=db1, dh=dh, dw1=dw1, dx=dx, dw=dw,
                dscale=dscale, dshift=dshift)


def near(got, want, slack):
    bound = slack + (_mx8.step_of(want, got.dtype) * (1 + 2.0 ** -10)
                     if got.dtype != torch.float32 else 2.0 ** -24 * want.abs())
    assert got.shape == want.shape and ((got.double() - want).abs() <= bound).all()


def test_step(rm):
    t = inputs(rm)
    g = step(rm, t)
    d = {k: _mx8.decoded(v) if isinstance(v, rm.Mxfp8) else v.double() for k, v in g.items()}
    f = {k: v.double() for k, v in t.items()}

    def product(a, b, bias=None):
        z = a @ b.T
        slack = (b.shape[1] / 32 + 2) * 2.0 ** -23 * (a.abs() @ b.abs().T)
        return (z, slack) if bias is None else (z + bias, slack + 2.0 ** -24 * (z + bias).abs())

    near(g["res"], f["x"] + f["update"], 2.0 ** -24 * (f["x"] + f["update"]).abs())
    r = (d["res"].square().mean(-1) + EPS).rsqrt()
    near(g["rstd"].view(B, S), r, 2.0 ** -20 * r)
    o = d["res"] * r[..., None] * f["weight"] * (1 + f["scale"])
    _mx8.check_held(g["h"], o + f["shift"], 2.0 ** -19 * (o.abs() + f["shift"].abs()))
    _mx8.check_held(g["kept"], d["res"], 0 * d["res"])
    z, s = product(d["h"], d["w1"], f["b1"])
    _mx8.check_held(g["z1"], z, s)
    y = _mx8.activation("gelu_tanh", z)[0]
    _mx8.check_held(g["a"], y, 1.2 * s + 2.0 ** -17 * y.abs() + 1e-30)
    z, s = product(d["a"], d["w2"], f["b2"])
    _mx8.check_held(g["z2"], z, s)
    y = d["res"] + f["gate"] * z
    near(g["y"], y, s * f["gate"].abs() + 2.0 ** -23 * (y.abs() + (f["gate"] * z).abs()))
    # backward
    dz = f["gy"] * f["gate"]
    _mx8.check_held(g["dz2"], dz, 2.0 ** -23 * dz.abs())
    n = (B * S + 8) * 2.0 ** -24
    near(g["db2"], dz.sum((0, 1)), n * dz.abs().sum((0, 1)))
    p = f["gy"] * d["z2"]
    near(g["dgate"], p.sum(1), n * p.abs().sum(1))

    def across(q):
        codes, e, _ = _mx8.shown(q)
        return torch.from_numpy(_mx8.values(*_mx8.across(codes, e))).cuda()

    near(g["da"], *product(d["dz2"], across(g["w2"])))
    near(g["dw2"], *product(across(g["dz2"]), across(g["a"])))
    h1, slope = _mx8.activation("gelu_tanh", d["z1"])
    dz = d["da"] * slope
    slack = 2.0 ** -20 * d["da"].abs() + 2.0 ** -22 * dz.abs()
    _mx8.check_held(g["dz1"], dz, slack)
    near(g["db1"], dz.sum((0, 1)), n * dz.abs().sum((0, 1)) + slack.sum((0, 1)))
    near(g["dh"], *product(d["dz1"], across(g["w1"])))
    near(g["dw1"], *product(across(g["dz1"]), across(g["h"])))
    rr = d["rstd"].view(B, S, 1)
    hh = d["kept"] * rr
    m = f["weight"] * (1 + f["scale"])
    u = d["dh"] * m
    dx = rr * (u - hh * (u * hh).mean(-1, keepdim=True)) + f["gy"]
    size = rr * (u.abs() + hh.abs() * (u * hh).abs().mean(-1, keepdim=True)) + f["gy"].abs()
    near(g["dx"], dx, (D / 32 + 16) * 2.0 ** -24 * size)
    p = d["dh"] * hh
    near(g["dw"], (p * (1 + f["scale"])).sum((0, 1)), n * (p * (1 + f["scale"])).abs().sum((0, 1)))
    near(g["dscale"], (p * f["weight"]).sum(1), n * (p * f["weight"]).abs().sum(1))
    near(g["dshift"], d["dh"].sum(1), n * d["dh"].abs().sum(1))


def bits(g):
    flat = []
    for v in g.values():
        flat += [v.codes.view(torch.uint8), v.scales] if isinstance(v, tuple) else [v]
    return [t.clone() for t in flat]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_step_on_another_stream(rm):
    t = inputs(rm, 1)
    want = bits(step(rm, t))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [step(rm, t, stream=side) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    assert all(same(bits(g), want) for g in got)
    with torch.cuda.stream(side):
        inside = step(rm, t)
    torch.cuda.current_stream().wait_stream(side)
    assert same(bits(inside), want)


def test_step_captured_and_replayed(rm):
    t, other = inputs(rm, 2), inputs(rm, 3)
    want = [bits(step(rm, t)), bits(step(rm, other))]
    static = {k: v.clone() for k, v in t.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(rm, static)  # first calls set kernels' attributes
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(rm, static)
        graphs.append((graph, out))
    for source, w in ((t, want[0]), (other, want[1]), (t, want[0])):
        for k, v in source.items():
            static[k].copy_(v)
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(same(bits(out), w) for _, out in graphs)


def test_empty_rows(rm):
    x = torch.zeros(2, 0, 64, dtype=torch.bfloat16, device="cuda")
    row = torch.ones(2, 1, 64, dtype=torch.bfloat16, device="cuda")
    rstd = torch.zeros(0, device="cuda")
    res, out, kept = rm.add_rmsnorm_mxfp8(x, x, None, row, row, keep=True)
    assert res.shape == out.codes.shape == kept.codes.shape == (2, 0, 64)
    gx, gw, gs, gh = rm.rmsnorm_mxfp8_backward(kept, row[0, 0], row, x, rstd)
    assert gx.shape == (2, 0, 64) and not gw.any() and not gs.any() and not gh.any()
    assert gs.shape == gh.shape == (2, 64)
    dz, db, dg = rm.mxfp8_activation_backward(kept, x, "silu", row)
    assert dz.codes.shape == (2, 0, 64) and not db.any() and not dg.any() and dg.shape == (2, 64)
    with pytest.raises(ValueError):
        rm.mxfp8_transpose(kept)


def test_gpu_refusals(rm):
    n = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    x = n(4, 64)
    q, w = rm.mxfp8_quantize(x), rm.mxfp8_quantize(n(16, 64))
    w32 = rm.mxfp8_quantize(n(32, 64))
    short = rm.Mxfp8(q.codes, q.scales[:256])
    for call in (
        lambda: rm.mxfp8_quantize(n(4, 48)), lambda: rm.mxfp8_quantize(n(64, 4).t()),
        lambda: rm.mxfp8_quantize(n(0)), lambda: rm.mxfp8_quantize(x, out=w),
        lambda: rm.mxfp8_dequantize(short), lambda: rm.mxfp8_dequantize(q, out=n(4, 32)),
        lambda: rm.mxfp8_transpose(q, out=w),
        lambda: rm.mxfp8_linear(x, w, bias=n(8)), lambda: rm.mxfp8_linear(x, w, gate=n(3, 1, 16)),
        lambda: rm.mxfp8_linear(x, w, residual=n(4, 8)), lambda: rm.mxfp8_linear(x, w, out=n(4, 8)),
        lambda: rm.mxfp8_linear(x, w, bias=torch.zeros(16, dtype=torch.bfloat16)),
        lambda: rm.mxfp8_linear(x, w, quantize=True), lambda: rm.mxfp8_linear(x, w, keep=True),
        lambda: rm.mxfp8_linear(x, w32, keep=q), lambda: rm.mxfp8_linear(x, w, activation="tanh"),
        lambda: rm.mxfp8_linear(x, w, activation=1), lambda: rm.mxfp8_linear(n(4, 96), w),
        lambda: rm.mxfp8_linear(x, rm.mxfp8_quantize(n(12, 64))),
        lambda: rm.mxfp8_linear(short, w),
        lambda: rm.mxfp8_activation_backward(q, n(4, 32)),
        lambda: rm.mxfp8_activation_backward(q, x, "relu"),
        lambda: rm.mxfp8_activation_backward(q, x, gate=n(3, 1, 64)),
        lambda: rm.mxfp8_activation_backward(q, x, workspace=n(16, t=torch.uint8)),
        lambda: rm.add_rmsnorm_mxfp8(n(4, 40)), lambda: rm.add_rmsnorm_mxfp8(x, res_out=x),
        lambda: rm.add_rmsnorm_mxfp8(x, n(3, 64)), lambda: rm.add_rmsnorm_mxfp8(x, weight=n(32)),
        lambda: rm.add_rmsnorm_mxfp8(x, scale=n(3, 64)), lambda: rm.add_rmsnorm_mxfp8(x, out=w),
        lambda: rm.add_rmsnorm_mxfp8(x, rstd_out=torch.zeros(3, device="cuda")),
        lambda: rm.rmsnorm_mxfp8_backward(q, None, None, x, None),
        lambda: rm.rmsnorm_mxfp8_backward(q, None, None, n(4, 32), torch.zeros(4, device="cuda")),
        lambda: rm.rmsnorm_mxfp8_backward(q, n(64), None, x, torch.zeros(4, device="cuda"),
                                          workspace=n(16, t=torch.uint8)),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: rm.mxfp8_linear(x, w, bias=n(16, t=torch.float16)),
        lambda: rm.mxfp8_linear(x, w, dtype=torch.float16),
        lambda: rm.mxfp8_linear(x, w, dtype=torch.float32),
        lambda: rm.mxfp8_linear(x, w32, out=n(4, 32), quantize=True),
        lambda: rm.add_rmsnorm_mxfp8(x, n(4, 64, t=torch.float16)),
        lambda: rm.mxfp8_activation_backward(q, x.float()),
    ):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(rm.RmsmodError):  # rows that start between two 16-byte vectors
        rm.mxfp8_quantize(n(4 * 64 + 4)[4:].view(4, 64))
    with pytest.raises(rm.RmsmodError):  # the result over a part of the residual
        buf = n(5, 16)
        rm.mxfp8_linear(x, w, residual=buf[:4], out=buf[1:])


def test_rows_on_16_bytes_only(rm):
    # tensors that start on 16 and not on 32 bytes give the same bits
    gen = torch.Generator(device="cuda").manual_seed(9)
    x, u, r = (torch.randn(150, 96, device="cuda", generator=gen).bfloat16() for _ in range(3))
    odd = lambda t: torch.cat([t.new_zeros(8), t.reshape(-1)])[8:].view(t.shape)  # noqa: E731
    odd8 = lambda q: rm.Mxfp8(torch.cat([q.codes.view(torch.uint8).new_zeros(16),  # noqa: E731
                                         q.codes.view(torch.uint8).reshape(-1)])[16:]
                              .view(torch.float8_e4m3fn).view(q.codes.shape), q.scales)
    assert odd(x).data_ptr() % 32 == 16
    a, b = rm.add_rmsnorm_mxfp8(x, u, keep=True), rm.add_rmsnorm_mxfp8(odd(x), odd(u), keep=True)
    assert torch.equal(a[0], b[0])
    for p, q in zip(a[1:], b[1:]):
        assert torch.equal(p.codes.view(torch.uint8), q.codes.view(torch.uint8))
    t, s = rm.mxfp8_transpose(a[1]), rm.mxfp8_transpose(odd8(a[1]))
    assert torch.equal(t.codes.view(torch.uint8), s.codes.view(torch.uint8))
    w = rm.mxfp8_quantize(torch.randn(96, 96, device="cuda", generator=gen).bfloat16())
    y = [rm.mxfp8_linear(f(a[1]), w, residual=g(r), out=g(torch.empty_like(r)),
                         keep=f(rm.mxfp8_quantize(r))) for f, g in ((lambda q: q, lambda t: t),
                                                                   (odd8, odd))]
    assert torch.equal(y[0][0], y[1][0])
    assert torch.equal(y[0][1].codes.view(torch.uint8), y[1][1].codes.view(torch.uint8))


def test_two_calls_share_their_inputs(rm):
    # two streams at once over the same inputs, each with results and workspace of its own
    t = inputs(rm, 5)
    want = bits(step(rm, t))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for s in streams:
            got.append(step(rm, t, stream=s))
    for s in streams:
        torch.cuda.current_stream().wait_stream(s)
    assert all(same(bits(g), want) for g in got)
