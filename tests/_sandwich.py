"""The norms after and before a block and their gradients from the definition, in float64.

Tensors [B, S, D]; row vectors None, [D], or [B or 1, 1, D].  Beside every value the magnitude of the
terms it is a sum of, which is what the rounding of an fp32 evaluation scales with."""
import torch


def d(t):
    return None if t is None else t.detach().double()


def factor(*ts):
    """Product of those that are there (1 without any)."""
    v = torch.ones((), dtype=torch.float64)
    for t in ts:
        if t is not None:
            v = v.to(t.device) * d(t)
    return v


def rstd(x, eps):
    return (d(x).square().mean(-1, keepdim=True) + eps).rsqrt()


def residual_add(residual, update, post_weight, gate, post_eps, residual_scale, update_scale):
    a = residual_scale * d(residual)
    b = d(update) * rstd(update, post_eps) * factor(post_weight, gate) * update_scale
    return a + b, a.abs() + b.abs()


def multiplier(weight, scale):
    return factor(weight, None if scale is None else 1.0 + d(scale))


def norm(res, weight, scale, shift, eps):
    a = d(res) * rstd(res, eps) * multiplier(weight, scale)
    b = 0.0 if shift is None else d(shift)
    return a + b, a.abs() + (b.abs() if shift is not None else 0.0)


def columns(t, rows):
    """Sums over the tokens: per batch (rows = B), or over the batches too (rows = 1)."""
    t = t.sum(1)
    return t if rows == t.shape[0] else t.sum(0, keepdim=True)


def norm_grad(res, weight, scale, go, gr, r, rows, got):
    """dh and its magnitude; the row vectors' gradients into `got`."""
    h, g = d(res) * r, d(go)
    gm = g * multiplier(weight, scale)
    dh = r * (gm - h * (gm * h).mean(-1, keepdim=True))
    size = r * (gm.abs() + h.abs() * (gm * h).abs().mean(-1, keepdim=True))
    if gr is not None:
        dh, size = dh + d(gr), size + d(gr).abs()
    w, one = factor(weight), multiplier(None, scale)
    got["shift"] = columns(g, rows), columns(g.abs(), rows)
    got["scale"] = columns(g * h * w, rows), columns((g * h * w).abs(), rows)
    got["weight"] = columns(g * h * one, 1)[0], columns((g * h * one).abs(), 1)[0]
    return dh, size


def sandwich_grad(update, res, post_weight, gate, weight, scale, gr, go, rp, r, residual_scale,
                  update_scale, mod_rows=1, gate_rows=1):
    """{name: (value, magnitude)}; rp, r [B, S, 1] float64."""
    got = {}
    if go is not None:
        dh, size = norm_grad(res, weight, scale, go, gr, r, mod_rows, got)
    else:
        dh, size = d(gr), d(gr).abs()
    got["residual"] = residual_scale * dh, abs(residual_scale) * size
    uh, v = d(update) * rp, factor(post_weight, gate) * update_scale
    dv, sv = dh * v, size * v.abs()
    got["update"] = (rp * (dv - uh * (dv * uh).mean(-1, keepdim=True)),
                     rp * (sv + uh.abs() * (sv * uh.abs()).mean(-1, keepdim=True)))
    p, q = dh * uh * update_scale, size * uh.abs() * abs(update_scale)
    wp, g = factor(post_weight), factor(gate)
    got["gate"] = columns(p * wp, gate_rows), columns(q * wp.abs(), gate_rows)
    got["post_weight"] = columns(p * g, 1)[0], columns(q * g.abs(), 1)[0]
    return got
