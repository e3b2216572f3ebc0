"""The sandwich norms without a GPU: the float64 reference against central differences and autograd,
workspace sizes, and every refusal (nothing launched)."""
import ctypes

import pytest
import torch

import _sandwich as ref

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_STRIDE, ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5
P = ctypes.c_void_p
A = 0x100000000


@pytest.fixture(scope="module")
def rm():
    from rmsnorm_modulate_gb300 import _build

    _build.build()
    import rmsnorm_modulate_gb300 as rm

    rm.library()
    return rm


@pytest.mark.parametrize("per_batch", [False, True])
def test_reference_gradients_against_differences(per_batch):
    gen = torch.Generator().manual_seed(1)
    B, S, D = 2, 3, 8
    rows = B if per_batch else 1
    n = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)  # noqa: E731
    t = dict(residual=n(B, S, D), update=n(B, S, D), post_weight=1 + 0.1 * n(D),
             gate=n(rows, 1, D), weight=1 + 0.1 * n(D), scale=0.3 * n(rows, 1, D),
             shift=n(rows, 1, D))
    gr, go, eps, rs, us = n(B, S, D), n(B, S, D), 1e-3, 0.7, 1.3

    def loss(t):
        res, _ = ref.residual_add(t["residual"], t["update"], t["post_weight"], t["gate"], eps, rs,
                                  us)
        out, _ = ref.norm(res, t["weight"], t["scale"], t["shift"], eps)
        return (res * gr).sum() + (out * go).sum()

    res, _ = ref.residual_add(t["residual"], t["update"], t["post_weight"], t["gate"], eps, rs, us)
    got = ref.sandwich_grad(t["update"], res, t["post_weight"], t["gate"], t["weight"], t["scale"],
                            gr, go, ref.rstd(t["update"], eps), ref.rstd(res, eps), rs, us, rows,
                            rows)
    step = 1e-5
    for name, x in t.items():
        want = torch.zeros(x.numel(), dtype=torch.float64)
        for i in range(x.numel()):
            ends = []
            for s in (step, -step):
                y = x.clone()
                y.view(-1)[i] += s
                ends.append(loss({**t, name: y}))
            want[i] = (ends[0] - ends[1]) / (2 * step)
        # third derivatives of order 1 to 100 times step^2, and 2^-52 of the loss over the step
        assert (got[name][0].reshape(-1) - want).abs().max() < 1e-7, name


def test_workspace_bytes(rm):
    lib = rm.library()
    f, g = (lib.sandwich_rmsnorm_modulate_backward_workspace_bytes,
            lib.rmsnorm_modulate_backward_workspace_bytes)
    for B, S, D in ((1, 1, 8), (2, 77, 1024), (3, 5000, 16384)):
        assert f(B, S, D) % (12 * D * B) == 0 and f(B, S, D) * 2 == g(B, S, D) * 3 > 0
        assert f(B, S, D) == B * f(1, S, D)  # the items of a batch do not depend on the others
    for B, S, D in ((0, 4, 64), (1, 0, 64), (1, 4, 12), (1, 4, 16392), (-1, 4, 64)):
        assert f(B, S, D) == 0 and g(B, S, D) == 0


def at(i):
    return A + (i << 24)


def test_forward_refusals(rm):
    f = rm.library().sandwich_rmsnorm_modulate

    def call(x=at(0), u=at(1), pw=at(2), g=at(3), gs=64, w=at(4), sc=at(5), sh=at(6), ms=64,
             ro=at(7), o=at(8), B=2, S=16, D=64, st=at(9), st2=at(10), dtype=0):
        return f(P(x), P(u), P(pw), P(g), gs, P(w), P(sc), P(sh), ms, P(ro), P(o), B, S, D, 1.0,
                 1.0, 1e-6, 1e-6, P(st), P(st2), dtype, P(0))

    for k in (dict(D=12), dict(D=0), dict(D=16392), dict(B=-1), dict(S=-1),
              dict(B=1 << 40, S=1 << 40)):
        assert call(**k) == ERR_SHAPE, k
    assert call(dtype=2) == ERR_UNSUPPORTED
    for k in (dict(gs=4), dict(ms=-8), dict(B=1 << 20, S=1, gs=1 << 60)):
        assert call(**k) == ERR_STRIDE, k
    assert call(S=0, x=0, u=0, ro=0) == OK and call(B=0) == OK
    for k in ("x", "u", "ro"):
        assert call(**{k: 0}) == ERR_NULL, k
    for k in ("x", "u", "pw", "g", "w", "sc", "sh", "ro", "o"):
        assert call(**{k: at(12) + 8}) == ERR_ALIGN, k
    for k in ("st", "st2"):
        assert call(**{k: at(12) + 2}) == ERR_ALIGN, k
    for out in ("ro", "o", "st", "st2"):
        for i in range(0 if out != "ro" else 1, 7):  # over any input (res over residual may be)
            assert call(**{out: at(i)}) == ERR_UNSUPPORTED, (out, i)
    assert call(ro=at(0) + 16) == ERR_UNSUPPORTED
    assert call(o=at(7)) == ERR_UNSUPPORTED and call(st=at(8)) == ERR_UNSUPPORTED
    assert call(st=at(9), st2=at(9) + 4) == ERR_UNSUPPORTED
    assert call(g=at(8) - 2 * 64, gs=64) == ERR_UNSUPPORTED  # the second gate row reaches into out


def test_backward_refusals(rm):
    f = rm.library().sandwich_rmsnorm_modulate_backward

    def call(u=at(0), h=at(1), pw=at(2), g=at(3), gs=64, w=at(4), sc=at(5), ms=64, gr=at(6),
             go=at(7), rp=at(8), r=at(9), B=2, S=16, D=64, gx=at(10), gu=at(11), gpw=at(12),
             gg=at(13), gw=at(14), gsc=at(15), gsh=at(16), ws=at(17), wb=1 << 20, dtype=0):
        return f(P(u), P(h), P(pw), P(g), gs, P(w), P(sc), ms, P(gr), P(go), P(rp), P(r), B, S, D,
                 1.0, 1.0, P(gx), P(gu), P(gpw), P(gg), P(gw), P(gsc), P(gsh), P(ws), wb, dtype,
                 P(0))

    for k in (dict(D=12), dict(B=-1), dict(S=-1), dict(D=16392), dict(wb=64)):
        assert call(**k) == ERR_SHAPE, k
    assert call(dtype=5) == ERR_UNSUPPORTED
    assert call(gs=4) == ERR_STRIDE and call(ms=-64) == ERR_STRIDE
    for k in ("u", "h", "rp", "r", "ws"):
        assert call(**{k: 0}) == ERR_NULL, k
    assert call(go=0, gr=0, gw=0, gsc=0, gsh=0) == ERR_NULL
    assert call(go=0) == ERR_UNSUPPORTED  # a weight's gradient without the norm it belongs to
    for k in ("u", "h", "pw", "g", "w", "sc", "gr", "go", "gx", "gu", "gpw", "gg", "gw", "gsc",
              "gsh"):
        assert call(**{k: at(20) + 8}) == ERR_ALIGN, k
    assert call(ws=at(20) + 16) == ERR_ALIGN and call(rp=at(20) + 2) == ERR_ALIGN
    assert call(gx=0, gu=0, gpw=0, gg=0, gw=0, gsc=0, gsh=0) == OK  # nothing wanted
    outs = ("gx", "gu", "gpw", "gg", "gw", "gsc", "gsh", "ws")
    for i, k in enumerate(outs):
        for j in range(10):
            assert call(**{k: at(j)}) == ERR_UNSUPPORTED, (k, j)
        for j in range(i):
            assert call(**{k: at(10 + j)}) == ERR_UNSUPPORTED, (k, j)


def test_rms_backward_refusals(rm):
    f = rm.library().rmsnorm_modulate_backward

    def call(x=at(0), w=at(1), sc=at(2), ms=64, go=at(3), gr=at(4), r=at(5), B=2, S=16, D=64,
             gx=at(6), gw=at(7), gsc=at(8), gsh=at(9), ws=at(10), wb=1 << 20):
        return f(P(x), P(w), P(sc), ms, P(go), P(gr), P(r), B, S, D, P(gx), P(gw), P(gsc), P(gsh),
                 P(ws), wb, P(0))

    assert call(D=20) == ERR_SHAPE and call(wb=0) == ERR_SHAPE and call(ms=4) == ERR_STRIDE
    for k in ("x", "go", "r", "ws"):
        assert call(**{k: 0}) == ERR_NULL, k
    assert call(go=at(12) + 8) == ERR_ALIGN
    for k in ("gx", "gw", "gsc", "gsh", "ws"):
        for j in range(6):
            assert call(**{k: at(j)}) == ERR_UNSUPPORTED, (k, j)
    assert call(gx=0, gw=0, gsc=0, gsh=0) == OK


def test_python_refusals(rm):
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        rm.sandwich_rmsnorm_modulate(x, x)  # no CPU path
    with pytest.raises(TypeError):
        rm.sandwich_rmsnorm_modulate(x.float(), x)
    with pytest.raises(ValueError):
        rm.rmsnorm_modulate_backward(x, None, None, x, None)
    with pytest.raises(ValueError):
        rm.sandwich_rmsnorm_modulate_backward(x, x, None, None, None, None, x, x, None, None)
