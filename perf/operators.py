"""The operators around a transformer block -- the norms before and after it fused with its gate
and residual scale, their gradients, and its projections in microscaled 4-bit floating point -- in
a plain form (elementary torch operations in 32 bits) and as calls of rmsnorm_modulate_gb300.

    sandwich  res = R(residual_scale * residual + update_scale * gate * RMSNorm(update) * post_weight)
              out = R(RMSNorm(res) * weight * (1 + scale) + shift)
    sandwich_grad   the gradients of that, given those of res and out
    rms_grad        the gradients of the norm before a block alone
    quantize        rows to blocks of 32 e2m1 values under one power-of-two scale, and back
    linear          the 4-bit product x w^T, with bias, gate and residual in its epilogue

`own` says which of the two forms run() takes.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
_EPS = 1e-6


def listed():
    return [
        # one token of each of four requests, each with its own adaLN rows: latency
        dict(name="sandwich_tokens_4x1x4096", op="sandwich", B=4, S=1, D=4096, dtype="bf16",
             per_batch=True, gated=True, mod=True, out=True, stats=False),
        # an image's tokens through one block boundary in training: statistics kept
        dict(name="sandwich_image_1x4216x4096", op="sandwich", B=1, S=4216, D=4096, dtype="bf16",
             per_batch=False, gated=True, mod=True, out=True, stats=True),
        # a language model's sandwich norms: no adaLN rows, wide, fp16, an odd length
        dict(name="sandwich_text_2x1777x6144_f16", op="sandwich", B=2, S=1777, D=6144,
             dtype="f16", per_batch=False, gated=False, mod=False, out=True, stats=False),
        # a short ragged text stream in training, per-sample adaLN rows
        dict(name="sandwich_grad_2x77x1024", op="sandwich_grad", B=2, S=77, D=1024, dtype="bf16",
             per_batch=True, gated=True, mod=True, out=True),
        # the training step's block boundary at an image's length
        dict(name="sandwich_grad_1x4216x4096", op="sandwich_grad", B=1, S=4216, D=4096,
             dtype="bf16", per_batch=False, gated=True, mod=True, out=True),
        # the first norm of a small model
        dict(name="rms_grad_1x256x1024", op="rms_grad", B=1, S=256, D=1024, dtype="bf16",
             per_batch=False, mod=True, stream=False),
        # the norm before the first block, a batch of two images, joined by the stream's gradient
        dict(name="rms_grad_2x4216x4096", op="rms_grad", B=2, S=4216, D=4096, dtype="bf16",
             per_batch=True, mod=True, stream=True),
        # a few tokens' activations
        dict(name="quantize_16x4096", op="quantize", M=16, K=4096, dtype="bf16"),
        # the input of a block's second projection at an image's length
        dict(name="quantize_4216x16384", op="quantize", M=4216, K=16384, dtype="bf16"),
        # a few tokens through a projection: the weights' bytes are what counts
        dict(name="linear_8x4096x4096", op="linear", B=1, S=8, N=4096, K=4096, dtype="bf16",
             bias=True, joined=False),
        # the first projection of a block's feed-forward part
        dict(name="linear_4216x16384x4096", op="linear", B=1, S=4216, N=16384, K=4096,
             dtype="bf16", bias=True, joined=False),
        # its second one, which ends in the gated residual add; two ragged samples
        dict(name="linear_2x2107x4096x16384", op="linear", B=2, S=2107, N=4096, K=16384,
             dtype="bf16", bias=False, joined=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _step(v, m):
    return max(m, v // m * m)


def draw(rng):
    op = rng.choice(["sandwich", "sandwich_grad", "rms_grad", "quantize", "linear"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "quantize":
        K = _step(_log(rng, 32, 16384), 32)
        return dict(op=op, M=_log(rng, 1, min(40000, 4216 * 16384 // K)), K=K, dtype=dtype)
    if op == "linear":
        K, N = _step(_log(rng, 64, 16384), 32), _step(_log(rng, 64, 16384), 8)
        B = rng.randint(1, 3)
        S = _log(rng, 1, min(4216, 4216 * 16384 * 4096 // (K * N)) // B)
        return dict(op=op, B=B, S=S, N=N, K=K, dtype=dtype, bias=rng.random() < 0.5,
                    joined=rng.random() < 0.5)
    D = _step(_log(rng, 256, 16384), 8)
    B = rng.randint(1, 4)
    S = _log(rng, 1, min(16384, 4216 * 4096 // D) // B)
    case = dict(op=op, B=B, S=S, D=D, dtype=dtype, per_batch=rng.random() < 0.5,
                mod=rng.random() < 0.7)
    if op == "rms_grad":
        return dict(case, dtype="bf16", stream=rng.random() < 0.5)
    case.update(gated=rng.random() < 0.7, out=rng.random() < 0.8)
    return dict(case, stats=rng.random() < 0.5) if op == "sandwich" else case


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _rms(x):
    return 1.0 / torch.sqrt(x.square().mean(-1) + _EPS)


def _stream(gen, B, S, D):
    """Activations with the outlier rows that a residual stream has."""
    x = torch.randn(B, S, D, device="cuda", generator=gen)
    return x * torch.where(torch.rand(B, S, 1, device="cuda", generator=gen) < 0.01, 20.0, 1.0)


def _blocks(gen, rows, K, dtype):
    """A 4-bit weight matrix as a checkpoint holds it: packed codes, and the scale bytes in tiles
    of 128 rows by 4 blocks (row r, block k of a tile at byte (r % 32) * 16 + r // 32 * 4 + k)."""
    packed = torch.randint(0, 256, (rows, K // 2), device="cuda", generator=gen,
                           dtype=torch.uint8)
    # weights of a layer of K inputs: entries of about 1 / sqrt(K)
    top = 127 - int(round(math.log2(3.0 * math.sqrt(K))))
    grid = torch.randint(top - 2, top + 2, (rows, K // 32), device="cuda", generator=gen,
                         dtype=torch.uint8)
    R, C = -(-rows // 128), -(-K // 128)
    full = torch.zeros(R * 128, C * 4, dtype=torch.uint8, device="cuda")
    full[:rows, :K // 32] = grid
    return packed, full.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = _TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std + mean).to(T)

    s = dict(case)
    if case["op"] == "quantize":
        s["x"] = _stream(gen, 1, case["M"], case["K"])[0].to(T)
        return s
    if case["op"] == "linear":
        B, S, N, K = case["B"], case["S"], case["N"], case["K"]
        s["x"] = normal(B, S, K)
        s["w"], s["w_scales"] = _blocks(gen, N, K, T)
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        s["residual"] = _stream(gen, B, S, N).to(T) if case["joined"] else None
        s["gate"] = normal(B, 1, N, std=0.1) if case["joined"] else None
        return s
    B, S, D = case["B"], case["S"], case["D"]
    rows = B if case["per_batch"] else 1
    # the adaLN projection's output, cut into gate, scale and shift: strided views
    cut = normal(rows, 1, 3 * D, std=0.1).chunk(3, dim=-1)
    s["weight"] = normal(D, std=0.05, mean=1.0)
    s["scale"], s["shift"] = (cut[1], cut[2]) if case["mod"] else (None, None)
    if case["op"] == "rms_grad":
        s["x"] = _stream(gen, B, S, D).to(T)
        s["rstd"] = _rms(s["x"].float()).view(-1)
        s["grad_out"] = normal(B, S, D)
        s["grad_res"] = normal(B, S, D) if case["stream"] else None
        return s
    s["update"] = _stream(gen, B, S, D).to(T)
    s["post_weight"] = normal(D, std=0.05, mean=1.0)
    s["gate"] = cut[0] if case["gated"] else None
    s["update_scale"] = 1.0 if case["gated"] else 0.25
    s["residual_scale"] = 1.0
    if not case["out"]:
        s["weight"] = s["scale"] = s["shift"] = None
    stream = _stream(gen, B, S, D).to(T)
    if case["op"] == "sandwich":
        s["residual"] = stream
        return s
    s["res"] = stream  # what the forward pass left
    s["post_rstd"] = _rms(s["update"].float()).view(-1)
    s["rstd"] = _rms(stream.float()).view(-1) if case["out"] else None
    s["grad_res"] = normal(B, S, D)
    s["grad_out"] = normal(B, S, D) if case["out"] else None
    return s


# ---------------------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------------------

def _f(t):
    return None if t is None else t.float()


def _plain_sandwich(s):
    T = s["update"].dtype
    u = s["update"].float()
    post_rstd = _rms(u)
    v = s["post_weight"].float() * s["update_scale"]
    if s["gate"] is not None:
        v = v * s["gate"].float()
    res = (s["residual"].float() * s["residual_scale"] + u * post_rstd[..., None] * v).to(T)
    got = {"res": res}
    if s["stats"]:
        got["post_rstd"] = post_rstd.reshape(-1)
    if s["out"]:
        h = res.float()
        rstd = _rms(h)
        o = h * rstd[..., None] * s["weight"].float()
        if s["mod"]:
            o = o * (1.0 + s["scale"].float()) + s["shift"].float()
        got["out"] = o.to(T)
        if s["stats"]:
            got["rstd"] = rstd.reshape(-1)
    return got


def _columns(t, per_batch):
    """Sums over the tokens, and over the batch where the row is shared."""
    return t.sum(1) if per_batch else t.sum((0, 1)).unsqueeze(0)


def _plain_norm_grad(s, h, got):
    """Gradients of out = h * rstd * weight * (1 + scale) + shift by h, and by the rows."""
    go, w = s["grad_out"].float(), s["weight"].float()
    rstd = s["rstd"].view(h.shape[0], h.shape[1], 1)
    hat = h * rstd
    m = w
    if s["mod"]:
        one = 1.0 + s["scale"].float()
        m = w * one
        got["grad_scale"] = _columns(go * hat * w, s["per_batch"])
        got["grad_shift"] = _columns(go, s["per_batch"])
        got["grad_weight"] = (go * hat * one).sum((0, 1))
    else:
        got["grad_weight"] = (go * hat).sum((0, 1))
    d = go * m
    return rstd * (d - hat * (d * hat).mean(-1, keepdim=True))


def _plain_sandwich_grad(s):
    T = s["update"].dtype
    got = {}
    dh = s["grad_res"].float()
    if s["out"]:
        dh = dh + _plain_norm_grad(s, s["res"].float(), got)
    got["grad_residual"] = (dh * s["residual_scale"]).to(T)
    r = s["post_rstd"].view(dh.shape[0], dh.shape[1], 1)
    hat = s["update"].float() * r
    wp = s["post_weight"].float() * s["update_scale"]
    v = wp
    if s["gate"] is not None:
        g = s["gate"].float()
        v = wp * g
        got["grad_gate"] = _columns(dh * hat * wp, s["per_batch"])
        got["grad_post_weight"] = (dh * hat * (g * s["update_scale"])).sum((0, 1))
    else:
        got["grad_post_weight"] = (dh * hat * s["update_scale"]).sum((0, 1))
    d = dh * v
    got["grad_update"] = (r * (d - hat * (d * hat).mean(-1, keepdim=True))).to(T)
    return got


def _plain_rms_grad(s):
    got = {}
    dx = _plain_norm_grad(s, s["x"].float(), got)
    if s["grad_res"] is not None:
        dx = dx + s["grad_res"].float()
    got["grad_x"] = dx.to(s["x"].dtype)
    return got


def _plain_rounded(x):
    """x [rows, K] rounded to e2m1 under the block scale 2^s, the least with amax <= 6 * 2^s."""
    b = x.float().view(x.shape[0], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    mant, e = torch.frexp(amax)  # amax = mant * 2^e, mant in [0.5, 1)
    e = torch.where(mant > 0.75, e - 2, e - 3).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    q = torch.ldexp(torch.ldexp(b, -(e // 2)), -(e - e // 2))
    a = q.abs()
    # the distance of neighbours: 0.5 below 2, 1 below 4, 2 from there on; ties to even
    unit = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0))
    q = torch.round(q / unit) * unit
    return torch.ldexp(torch.ldexp(q, e // 2), e - e // 2).view(x.shape)


def _plain_weights(packed, scales, K):
    rows = packed.shape[0]
    R, C = -(-rows // 128), -(-K // 128)
    grid = scales.view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, C * 4)
    grid = grid[:rows, :K // 32].int() - 127
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0,
                          -3.0, -4.0, -6.0], device=packed.device)
    codes = torch.stack([packed & 15, packed >> 4], dim=-1).view(rows, K // 32, 32)
    return torch.ldexp(table[codes.int()], grid[..., None]).view(rows, K)


def _plain_linear(s):
    B, S, N, K = s["B"], s["S"], s["N"], s["K"]
    y = _plain_rounded(s["x"].view(B * S, K)) @ _plain_weights(s["w"], s["w_scales"], K).t()
    y = y.view(B, S, N)
    if s["bias"] is not None:
        y = y + s["bias"].float()
    if s["joined"]:
        y = s["residual"].float() + s["gate"].float() * y
    return y.to(s["x"].dtype)


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------

def _own_sandwich(s):
    import rmsnorm_modulate_gb300 as rm

    post_rstd = rstd = None
    if s["stats"]:
        n = s["B"] * s["S"]
        post_rstd = torch.empty(n, dtype=torch.float32, device="cuda")
        rstd = torch.empty(n, dtype=torch.float32, device="cuda") if s["out"] else None
    res, out = rm.sandwich_rmsnorm_modulate(
        s["residual"], s["update"], s["post_weight"], s["gate"], s["weight"], s["scale"],
        s["shift"], eps=_EPS, post_eps=_EPS, residual_scale=s["residual_scale"],
        update_scale=s["update_scale"], need_out=s["out"], post_rstd_out=post_rstd,
        rstd_out=rstd)
    got = {"res": res}
    if s["out"]:
        got["out"] = out
    if s["stats"]:
        got["post_rstd"] = post_rstd
        if s["out"]:
            got["rstd"] = rstd
    return got


def _own_sandwich_grad(s):
    import rmsnorm_modulate_gb300 as rm

    g = rm.sandwich_rmsnorm_modulate_backward(
        s["update"], s["res"], s["post_weight"], s["gate"], s["weight"], s["scale"],
        s["grad_res"], s["grad_out"], s["post_rstd"], s["rstd"],
        residual_scale=s["residual_scale"], update_scale=s["update_scale"])
    got = {"grad_residual": g.residual, "grad_update": g.update,
           "grad_post_weight": g.post_weight}
    if s["gate"] is not None:
        got["grad_gate"] = g.gate
    if s["out"]:
        got["grad_weight"] = g.weight
        if s["mod"]:
            got["grad_scale"], got["grad_shift"] = g.scale, g.shift
    return got


def _own_rms_grad(s):
    import rmsnorm_modulate_gb300 as rm

    gx, gw, gsc, gsh = rm.rmsnorm_modulate_backward(
        s["x"], s["weight"], s["scale"], s["grad_out"], s["rstd"], grad_res=s["grad_res"])
    got = {"grad_x": gx, "grad_weight": gw}
    if s["mod"]:
        got["grad_scale"], got["grad_shift"] = gsc, gsh
    return got


def _own_quantize(s):
    import rmsnorm_modulate_gb300 as rm

    return rm.mxfp4_dequantize(rm.mxfp4_quantize(s["x"]), dtype=s["x"].dtype)


def _own_linear(s):
    import rmsnorm_modulate_gb300 as rm

    return rm.mxfp4_linear(s["x"], rm.Mxfp4(s["w"], s["w_scales"]), bias=s["bias"],
                           gate=s["gate"], residual=s["residual"])


def run(state):
    op = state["op"]
    if own:
        return {"sandwich": _own_sandwich, "sandwich_grad": _own_sandwich_grad,
                "rms_grad": _own_rms_grad, "quantize": _own_quantize,
                "linear": _own_linear}[op](state)
    if op == "quantize":
        return _plain_rounded(state["x"]).to(state["x"].dtype)
    return {"sandwich": _plain_sandwich, "sandwich_grad": _plain_sandwich_grad,
            "rms_grad": _plain_rms_grad, "linear": _plain_linear}[op](state)


def work(case):
    """Bytes of every input read once and every output written once, and the operations."""
    op = case["op"]
    if op == "quantize":  # rows in, 4-bit values and scales out and in again, values out
        n = case["M"] * case["K"]
        return {"bytes": 4 * n + 2 * (n // 2 + n // 32), "flops": 4 * n}
    if op == "linear":
        M, N, K = case["B"] * case["S"], case["N"], case["K"]
        b = 2 * M * K + N * (K // 2 + K // 32) + 2 * M * N
        if case["bias"]:
            b += 2 * N
        if case["joined"]:
            b += 2 * M * N + 2 * case["B"] * N
        return {"bytes": b, "flops": 2 * M * N * K}
    B, S, D = case["B"], case["S"], case["D"]
    rows, n = (B if case["per_batch"] else 1), B * S * D
    if op == "sandwich":
        tensors = 4 if case["out"] else 3
        cols = 1 + (rows if case["gated"] else 0)
        if case["out"]:
            cols += 1 + (2 * rows if case["mod"] else 0)
        stats = (2 if case["out"] else 1) * 4 * B * S if case["stats"] else 0
        return {"bytes": 2 * n * tensors + 2 * D * cols + stats,
                "flops": n * (14 if case["out"] else 7)}
    if op == "sandwich_grad":
        # in: update and the stream's gradient, res and out's gradient; out: two gradients
        tensors = 6 if case["out"] else 4
        cols = 2 + (2 * rows if case["gated"] else 0)
        cols_out = 1 + (rows if case["gated"] else 0)
        if case["out"]:
            cols += 1 + (rows if case["mod"] else 0)
            cols_out += 1 + (2 * rows if case["mod"] else 0)
        return {"bytes": 2 * n * tensors + 2 * D * cols + 4 * D * cols_out + 8 * B * S,
                "flops": n * (30 if case["out"] else 15)}
    tensors = 4 if case["stream"] else 3
    mod = rows if case["mod"] else 0
    return {"bytes": 2 * n * tensors + 2 * D * (1 + mod) + 4 * D * (1 + 2 * mod) + 4 * B * S,
            "flops": 15 * n}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_codes(x):
    """Nearest e2m1 value under the least power of two that holds the block, by search among the
    eight magnitudes; of two as near, the one whose code is even."""
    mags = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64,
                        device=x.device)
    b = x.double().reshape(-1, 32)
    got = torch.empty_like(b)
    for i in range(0, b.shape[0], 1 << 18):
        c = b[i:i + (1 << 18)]
        top = c.abs().max(-1, keepdim=True).values
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.ones_like(top)) / 6.0))
        # log2 may be off by its last bit at a border: settle it by products
        e = torch.where(6.0 * torch.exp2(e - 1) >= top, e - 1, e)
        e = torch.where(6.0 * torch.exp2(e) < top, e + 1, e)
        scale = torch.exp2(torch.where(top > 0, e, torch.full_like(e, -127.0)).clamp(min=-127.0))
        a = (c / scale).abs()
        lower = (torch.searchsorted(mags, a.contiguous(), right=True) - 1).clamp(0, 7)
        upper = (lower + 1).clamp(max=7)
        down, up = a - mags[lower], mags[upper] - a
        take = torch.where(down == up, lower + lower % 2, torch.where(down < up, lower, upper))
        got[i:i + (1 << 18)] = torch.copysign(mags[take.clamp(max=7)], c) * scale
    return got.view(x.shape)


def _exact_matrix(packed, scales, K):
    rows = packed.shape[0]
    r = torch.arange(rows, device=packed.device)[:, None]
    k = torch.arange(K // 32, device=packed.device)[None]
    tile = (r // 128) * (-(-K // 128)) + k // 4
    byte = scales[tile * 512 + r % 32 * 16 + r % 128 // 32 * 4 + k % 4]
    scale = torch.exp2(byte.double() - 127.0).repeat_interleave(32, dim=1)
    code = torch.empty(rows, K, dtype=torch.int64, device=packed.device)
    code[:, 0::2], code[:, 1::2] = packed % 16, packed // 16
    e, m = code % 8 // 2, code % 2
    mag = torch.where(e == 0, 0.5 * m, (1.0 + 0.5 * m) * torch.exp2(e.double() - 1.0))
    return torch.where(code >= 8, -mag, mag).double() * scale


def _rows64(t, B, fill):
    """Modulation rows as [B, 1, D] in 64 bits; `fill` where there are none."""
    return fill if t is None else t.double().reshape(-1, 1, t.shape[-1]).expand(B, 1, -1)


def _grad64(g, x, rstd, m):
    """Gradient of x * rstd(x) * m by x for the gradient g of the result."""
    n = x.shape[-1]
    dot = torch.einsum("bsd,bsd->bs", g * m, x)[..., None]
    return g * m * rstd - x * (rstd ** 3) * dot / n


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_codes(s["x"])
    if op == "linear":
        B, S, N, K = case["B"], case["S"], case["N"], case["K"]
        y = torch.matmul(_exact_codes(s["x"]).view(B * S, K),
                         _exact_matrix(s["w"], s["w_scales"], K).t()).view(B, S, N)
        if case["bias"]:
            y += s["bias"].double()
        if case["joined"]:
            y = torch.addcmul(s["residual"].double(), s["gate"].double(), y)
        return y
    B, S, D = case["B"], case["S"], case["D"]
    one = torch.ones(1, 1, D, dtype=torch.float64, device="cuda")
    scale1 = 1.0 + _rows64(s["scale"], B, 0.0 * one)
    w = one if s["weight"] is None else s["weight"].double() * one

    def fold(t, shared):
        t = torch.einsum("bsd->bd", t)
        return t.sum(0, keepdim=True) if shared else t

    if op == "sandwich":
        u, x = s["update"].double(), s["residual"].double()
        v = _rows64(s["gate"], B, one) * s["post_weight"].double() * s["update_scale"]
        r = (torch.einsum("bsd,bsd->bs", u, u) / D + _EPS).rsqrt()
        res = s["residual_scale"] * x + v * u * r[..., None]
        got = {"res": res}
        if case["stats"]:
            got["post_rstd"] = r.view(-1)
        if case["out"]:
            h = res.to(s["update"].dtype).double()
            r = (torch.einsum("bsd,bsd->bs", h, h) / D + _EPS).rsqrt()
            got["out"] = w * scale1 * h * r[..., None] + _rows64(s["shift"], B, 0.0 * one)
            if case["stats"]:
                got["rstd"] = r.view(-1)
        return got
    got = {}
    shared = not case["per_batch"]
    h = s["x" if op == "rms_grad" else "res"].double()
    dh = torch.zeros_like(h) if s["grad_res"] is None else s["grad_res"].double()
    if s["grad_out"] is not None:
        r = s["rstd"].double().view(B, S, 1)
        go = s["grad_out"].double()
        dh = dh + _grad64(go, h, r, w * scale1)
        p = go * h * r
        got["grad_weight"] = fold(p * scale1, True)[0]
        if case["mod"]:
            got["grad_scale"] = fold(p * w, shared)
            got["grad_shift"] = fold(go, shared)
    if op == "rms_grad":
        got["grad_x"] = dh
        return got
    got["grad_residual"] = dh * s["residual_scale"]
    gate = _rows64(s["gate"], B, one)
    wp = s["post_weight"].double() * one
    u, r = s["update"].double(), s["post_rstd"].double().view(B, S, 1)
    got["grad_update"] = _grad64(dh, u, r, gate * wp * s["update_scale"])
    p = dh * u * r * s["update_scale"]
    got["grad_post_weight"] = fold(p * gate, True)[0]
    if s["gate"] is not None:
        got["grad_gate"] = fold(p * wp, shared)
    return got
