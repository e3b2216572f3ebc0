"""A transformer block's projections in microscaled 8-bit floating point (blocks of 32 e4m3 codes
under one power-of-two scale), trained and served: the norm that feeds them, their product, and the
8-bit checkpoints that the backward pass takes its activations from -- in a plain form (elementary
torch operations in 32 bits) and as calls of rmsnorm_modulate_gb300.

    norm         res = R(x + update), out = Q(RMSNorm(res) * weight * (1 + scale) + shift), and
                 Q(res) for the backward pass
    linear       z = x w^T + bias, y = residual + gate * act(z) as R(y) or Q(y), and Q(z) for the
                 backward pass
    act_grad     Q(grad * gate * act'(z)) from the checkpoint z; its column sums (the bias's
                 gradient) and those of grad * act(z) (the gate's)
    norm_grad    the norm's gradients, from the checkpoint of its input
    weight_grad  grad_z^T x from 8-bit rows, laid out anew in blocks along the tokens, added to the
                 gradient so far

Q(v): 8-bit blocks; what is held in them is returned as the values it stands for.  `own` says which
of the two forms run() takes.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_EPS = 1e-6


def listed():
    return [
        # one token of each of four requests, each with its own adaLN rows: latency
        dict(name="norm_tokens_4x1x4096", op="norm", B=4, S=1, D=4096, dtype="bf16",
             per_batch=True, mod=True, update=True, keep=False),
        # an image's tokens before a block's first projection, in training: checkpoint, statistics
        dict(name="norm_image_1x4216x4096", op="norm", B=1, S=4216, D=4096, dtype="bf16",
             per_batch=False, mod=True, update=True, keep=True),
        # a language model's norm: no adaLN rows, wide, fp16, an odd length
        dict(name="norm_text_2x1777x6144_f16", op="norm", B=2, S=1777, D=6144, dtype="f16",
             per_batch=False, mod=False, update=True, keep=False),
        # a few tokens through a projection: the weights' bytes are what counts
        dict(name="linear_8x4096x4096", op="linear", B=1, S=8, N=4096, K=4096, dtype="bf16",
             x8=False, bias=True, act="silu", joined=False, quantize=False, keep=False),
        # the first projection of a block's feed-forward part, in training: its result feeds the
        # second one in 8 bits, what its activation saw is kept
        dict(name="linear_4216x16384x4096", op="linear", B=1, S=4216, N=16384, K=4096,
             dtype="bf16", x8=True, bias=True, act="gelu_tanh", joined=False, quantize=True,
             keep=True),
        # the second one, which ends in the gated residual add; two ragged samples
        dict(name="linear_2x2107x4096x16384", op="linear", B=2, S=2107, N=4096, K=16384,
             dtype="bf16", x8=True, bias=True, act="none", joined=True, quantize=False,
             keep=False),
        # the activation of a short ragged text stream, and its gated branch, in training
        dict(name="act_grad_2x77x4096", op="act_grad", B=2, S=77, N=4096, dtype="bf16",
             act="silu", gated=True, per_batch=True),
        # the activation of a feed-forward part at an image's length
        dict(name="act_grad_1x4216x16384", op="act_grad", B=1, S=4216, N=16384, dtype="bf16",
             act="gelu_tanh", gated=False, per_batch=False),
        # the norm of a short ragged text stream
        dict(name="norm_grad_2x77x1024", op="norm_grad", B=2, S=77, D=1024, dtype="bf16",
             per_batch=True, mod=True, stream=True),
        # the norm at an image's length, joined by the stream's gradient
        dict(name="norm_grad_1x4216x4096", op="norm_grad", B=1, S=4216, D=4096, dtype="bf16",
             per_batch=False, mod=True, stream=True),
        # a short stream's projection, added to the gradient of earlier micro-batches
        dict(name="weight_grad_154x4096x1024", op="weight_grad", T=154, N=4096, K=1024,
             added=True),
        # the first projection's weights at an image's length
        dict(name="weight_grad_4216x16384x4096", op="weight_grad", T=4216, N=16384, K=4096,
             added=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _step(v, m):
    return max(m, v // m * m)


def draw(rng):
    op = rng.choice(["norm", "linear", "act_grad", "norm_grad", "weight_grad"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "weight_grad":
        N, K = _step(_log(rng, 64, 16384), 32), _step(_log(rng, 64, 16384), 32)
        T = _log(rng, 1, min(4216, 4216 * 16384 * 4096 // (N * K)))
        return dict(op=op, T=T, N=N, K=K, added=rng.random() < 0.5)
    B = rng.randint(1, 4)
    if op == "linear":
        quantize, keep = rng.random() < 0.4, rng.random() < 0.4
        K = _step(_log(rng, 64, 16384), 32)
        N = _step(_log(rng, 64, 16384), 32 if quantize or keep else 8)
        most = min(4216, 4216 * 16384 * 4096 // (K * N))
        return dict(op=op, B=B, S=_log(rng, 1, max(1, most // B)), N=N, K=K, dtype=dtype,
                    x8=rng.random() < 0.6, bias=rng.random() < 0.6,
                    act=rng.choice(["none", "silu", "gelu", "gelu_tanh"]),
                    joined=rng.random() < 0.5, quantize=quantize, keep=keep)
    if op == "act_grad":
        N = _step(_log(rng, 64, 16384), 32)
        S = _log(rng, 1, min(16384, 4216 * 16384 // N) // B)
        return dict(op=op, B=B, S=S, N=N, dtype=dtype,
                    act=rng.choice(["none", "silu", "gelu", "gelu_tanh"]),
                    gated=rng.random() < 0.5, per_batch=rng.random() < 0.5)
    D = _step(_log(rng, 256, 16384), 32)
    S = _log(rng, 1, min(16384, 4216 * 4096 // D) // B)
    case = dict(op=op, B=B, S=S, D=D, dtype=dtype, per_batch=rng.random() < 0.5,
                mod=rng.random() < 0.7)
    if op == "norm_grad":
        return dict(case, stream=rng.random() < 0.7)
    return dict(case, update=rng.random() < 0.8, keep=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _rms(x):
    return 1.0 / torch.sqrt(x.square().mean(-1) + _EPS)


def _stream(gen, *shape):
    """Activations with the outlier rows that a residual stream has."""
    x = torch.randn(*shape, device="cuda", generator=gen)
    return x * torch.where(torch.rand(*shape[:-1], 1, device="cuda", generator=gen) < 0.01, 20.0,
                           1.0)


def _exponents(b):
    """Of blocks b [..., 32]: the least e with max|b| <= 448 * 2^e, at least -127."""
    amax = b.abs().amax(-1, keepdim=True)
    mant, e = torch.frexp(amax)  # amax = mant * 2^e, mant in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(mant > 0.875, e - 8, e - 9).clamp(min=-127)
    return torch.where(amax > 0, e, torch.full_like(e, -127))


def _scaled(v, e):
    """v * 2^e, in two steps that each stay in range."""
    return torch.ldexp(torch.ldexp(v, e // 2), e - e // 2)


def _held(x):
    """A matrix [rows, K] as 8-bit rows are kept: e4m3 codes, and the scale bytes in tiles of 128
    rows by 4 blocks (row r, block k of a tile at byte (r % 32) * 16 + r // 32 * 4 + k)."""
    rows, K = x.shape
    b = x.float().view(rows, -1, 32)
    e = _exponents(b)
    codes = _scaled(b, -e).view(rows, K).to(torch.float8_e4m3fn)
    R, C = -(-rows // 128), -(-K // 128)
    full = torch.zeros(R * 128, C * 4, dtype=torch.uint8, device=x.device)
    full[:rows, :K // 32] = (e[..., 0] + 127).to(torch.uint8)
    return codes, full.view(R, 4, 32, C, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = _TYPES[case.get("dtype", "f32")]

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, device="cuda", generator=gen) * std + mean).to(T)

    s = dict(case)
    op = case["op"]
    if op == "weight_grad":
        n, N, K = case["T"], case["N"], case["K"]
        # a loss's gradient: small, and of another size in each token
        size = torch.exp2(torch.randn(n, 1, device="cuda", generator=gen) - 12.0)
        s["grad_z"], s["grad_z_scales"] = _held(normal(n, N) * size)
        s["x"], s["x_scales"] = _held(normal(n, K))
        s["grad"] = normal(N, K, std=1e-3) if case["added"] else None
        return s
    B, S = case["B"], case["S"]
    if op == "linear":
        N, K = case["N"], case["K"]
        s["x"], s["x_scales"] = normal(B, S, K), None
        if case["x8"]:
            codes, s["x_scales"] = _held(s["x"].view(B * S, K))
            s["x"] = codes.view(B, S, K)
        s["w"], s["w_scales"] = _held(normal(N, K).float() / math.sqrt(K))
        s["bias"] = normal(N, std=0.1) if case["bias"] else None
        s["residual"] = _stream(gen, B, S, N).to(T) if case["joined"] else None
        s["gate"] = normal(B, 1, N, std=0.1) if case["joined"] else None
        return s
    if op == "act_grad":
        N = case["N"]
        codes, s["z_scales"] = _held(normal(B * S, N))
        s["z"] = codes.view(B, S, N)
        s["grad_out"] = normal(B, S, N)
        # the adaLN projection's output, cut into three: a strided view
        s["gate"] = normal(B if case["per_batch"] else 1, 1, 3 * N,
                           std=0.1).chunk(3, dim=-1)[1] if case["gated"] else None
        return s
    D = case["D"]
    cut = normal(B if case["per_batch"] else 1, 1, 2 * D, std=0.1).chunk(2, dim=-1)
    s["weight"] = normal(D, std=0.05, mean=1.0)
    s["scale"], s["shift"] = cut if case["mod"] else (None, None)
    x = _stream(gen, B, S, D).to(T)
    if op == "norm":
        s["x"] = x
        s["update"] = normal(B, S, D) if case["update"] else None
        return s
    s["rstd"] = _rms(x.float()).view(-1)  # what the forward pass left
    codes, s["kept_scales"] = _held(x.view(B * S, D))
    s["kept"] = codes.view(B, S, D)
    s["grad_out"] = normal(B, S, D)
    s["grad_res"] = normal(B, S, D) if case["stream"] else None
    return s


# ---------------------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------------------

def _rounded(x):
    """x [..., K] in fp32 as the 8-bit blocks hold it."""
    b = x.view(*x.shape[:-1], -1, 32)
    e = _exponents(b)
    return _scaled(_scaled(b, -e).to(torch.float8_e4m3fn).float(), e).view(x.shape)


def _values(codes, scales):
    """What 8-bit rows [..., K] stand for, in fp32."""
    K = codes.shape[-1]
    v = codes.float().view(-1, K // 32, 32)
    R, C = -(-v.shape[0] // 128), -(-K // 128)
    grid = scales.view(R, C, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R * 128, C * 4)
    e = grid[:v.shape[0], :K // 32, None].int() - 127
    return _scaled(v, e).view(codes.shape)


def _act(name, z):
    """-> act(z) and its derivative."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "gelu":
        half = 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
        return z * half, half + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if name == "silu":
        a, slope = z, 1.0
    else:  # 0.5 z (1 + tanh(a / 2)) = z sigmoid(a)
        c = 2.0 * math.sqrt(2.0 / math.pi)
        a, slope = c * (z + 0.044715 * z * z * z), c * (1.0 + 3.0 * 0.044715 * z * z)
    p = 1.0 / (1.0 + torch.exp(-a))
    return z * p, p + z * p * (1.0 - p) * slope


def _plain_norm(s):
    T = s["x"].dtype
    res = s["x"] if s["update"] is None else (s["x"].float() + s["update"].float()).to(T)
    h = res.float()
    rstd = _rms(h)
    o = h * rstd[..., None] * s["weight"].float()
    if s["mod"]:
        o = o * (1.0 + s["scale"].float()) + s["shift"].float()
    got = {"out": _rounded(o).to(T)}
    if s["update"] is not None:
        got["res"] = res
    if s["keep"]:
        got["kept"], got["rstd"] = _rounded(h).to(T), rstd.view(-1)
    return got


def _plain_linear(s):
    T = _TYPES[s["dtype"]]
    B, S, N, K = s["B"], s["S"], s["N"], s["K"]
    x = _values(s["x"], s["x_scales"]) if s["x8"] else _rounded(s["x"].float())
    z = (x.view(B * S, K) @ _values(s["w"], s["w_scales"]).t()).view(B, S, N)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    got = {}
    if s["keep"]:
        got["kept"] = _rounded(z).to(T)
    y = _act(s["act"], z)[0]
    if s["joined"]:
        y = s["residual"].float() + s["gate"].float() * y
    got["out"] = (_rounded(y) if s["quantize"] else y).to(T)
    return got


def _plain_act_grad(s):
    z = _values(s["z"], s["z_scales"])
    g = s["grad_out"].float()
    h, slope = _act(s["act"], z)
    got = {}
    dz = g * slope
    if s["gate"] is not None:
        dz = dz * s["gate"].float()
        t = g * h
        got["grad_gate"] = t.sum(1) if s["per_batch"] else t.sum((0, 1)).unsqueeze(0)
    got["grad_bias"] = dz.sum((0, 1))
    got["grad_z"] = _rounded(dz).to(s["grad_out"].dtype)
    return got


def _plain_norm_grad(s):
    h = _values(s["kept"], s["kept_scales"])
    go, w = s["grad_out"].float(), s["weight"].float()
    rstd = s["rstd"].view(h.shape[0], h.shape[1], 1)
    hat = h * rstd
    got = {}
    m = w
    if s["mod"]:
        one = 1.0 + s["scale"].float()
        m = w * one
        cols = (lambda t: t.sum(1)) if s["per_batch"] else (lambda t: t.sum((0, 1)).unsqueeze(0))
        got["grad_scale"], got["grad_shift"] = cols(go * hat * w), cols(go)
        got["grad_weight"] = (go * hat * one).sum((0, 1))
    else:
        got["grad_weight"] = (go * hat).sum((0, 1))
    d = go * m
    dx = rstd * (d - hat * (d * hat).mean(-1, keepdim=True))
    if s["grad_res"] is not None:
        dx = dx + s["grad_res"].float()
    got["grad_x"] = dx.to(s["grad_out"].dtype)
    return got


def _plain_across(codes, scales):
    """Rows' values [T, K] in blocks along the rows: [K, T up to a multiple of 32]."""
    v = _values(codes, scales).t()
    short = -v.shape[1] % 32
    if short:
        v = torch.cat([v, v.new_zeros(v.shape[0], short)], dim=1)
    return _rounded(v.contiguous())


def _plain_weight_grad(s):
    g = _plain_across(s["grad_z"], s["grad_z_scales"]) @ \
        _plain_across(s["x"], s["x_scales"]).t()
    return g if s["grad"] is None else s["grad"] + g


# ---------------------------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------------------------

def _own_norm(s):
    import rmsnorm_modulate_gb300 as rm

    T = s["x"].dtype
    rstd = torch.empty(s["B"] * s["S"], dtype=torch.float32, device="cuda") if s["keep"] else None
    res, out, kept = rm.add_rmsnorm_mxfp8(s["x"], s["update"], s["weight"], s["scale"], s["shift"],
                                          eps=_EPS, keep=s["keep"], rstd_out=rstd)
    got = {"out": rm.mxfp8_dequantize(out, dtype=T)}
    if s["update"] is not None:
        got["res"] = res
    if s["keep"]:
        got["kept"], got["rstd"] = rm.mxfp8_dequantize(kept, dtype=T), rstd
    return got


def _own_linear(s):
    import rmsnorm_modulate_gb300 as rm

    T = _TYPES[s["dtype"]]
    y = rm.mxfp8_linear(rm.Mxfp8(s["x"], s["x_scales"]) if s["x8"] else s["x"],
                        rm.Mxfp8(s["w"], s["w_scales"]), bias=s["bias"],
                        activation=None if s["act"] == "none" else s["act"], gate=s["gate"],
                        residual=s["residual"], dtype=T, quantize=s["quantize"], keep=s["keep"])
    got = {}
    if s["keep"]:
        y, kept = y
        got["kept"] = rm.mxfp8_dequantize(kept, dtype=T)
    got["out"] = rm.mxfp8_dequantize(y, dtype=T) if s["quantize"] else y
    return got


def _own_act_grad(s):
    import rmsnorm_modulate_gb300 as rm

    grad_z, grad_bias, grad_gate = rm.mxfp8_activation_backward(
        rm.Mxfp8(s["z"], s["z_scales"]), s["grad_out"],
        activation=None if s["act"] == "none" else s["act"], gate=s["gate"])
    got = {"grad_z": rm.mxfp8_dequantize(grad_z, dtype=s["grad_out"].dtype),
           "grad_bias": grad_bias}
    if s["gate"] is not None:
        got["grad_gate"] = grad_gate
    return got


def _own_norm_grad(s):
    import rmsnorm_modulate_gb300 as rm

    gx, gw, gsc, gsh = rm.rmsnorm_mxfp8_backward(
        rm.Mxfp8(s["kept"], s["kept_scales"]), s["weight"], s["scale"], s["grad_out"], s["rstd"],
        grad_res=s["grad_res"])
    got = {"grad_x": gx, "grad_weight": gw}
    if s["mod"]:
        got["grad_scale"], got["grad_shift"] = gsc, gsh
    return got


def _own_weight_grad(s):
    import rmsnorm_modulate_gb300 as rm

    return rm.mxfp8_linear(rm.mxfp8_transpose(rm.Mxfp8(s["grad_z"], s["grad_z_scales"])),
                           rm.mxfp8_transpose(rm.Mxfp8(s["x"], s["x_scales"])),
                           residual=s["grad"], dtype=torch.float32)


def run(state):
    op = state["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "act_grad": _own_act_grad,
                "norm_grad": _own_norm_grad, "weight_grad": _own_weight_grad}[op](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "act_grad": _plain_act_grad,
            "norm_grad": _plain_norm_grad, "weight_grad": _plain_weight_grad}[op](state)


def work(case):
    """Bytes of every input read once and every output written once, and the operations.  An 8-bit
    result (33 bytes to a block) is written, read again and returned as values of 16 bits."""
    op = case["op"]

    def held(n):
        return n + n // 32

    def shown(n):
        return 2 * held(n) + 2 * n

    if op == "weight_grad":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": held(T * N) + held(T * K) + 4 * N * K * (2 if case["added"] else 1),
                "flops": 2 * T * N * K}
    B, S = case["B"], case["S"]
    if op == "linear":
        M, N, K = B * S, case["N"], case["K"]
        b = (held(M * K) if case["x8"] else 2 * M * K) + held(N * K)
        b += shown(M * N) if case["quantize"] else 2 * M * N
        b += shown(M * N) if case["keep"] else 0
        b += 2 * N if case["bias"] else 0
        b += 2 * M * N + 2 * B * N if case["joined"] else 0
        return {"bytes": b, "flops": 2 * M * N * K}
    rows = B if case["per_batch"] else 1
    if op == "act_grad":
        n, N = B * S * case["N"], case["N"]
        return {"bytes": held(n) + 2 * n + shown(n) + 4 * N +
                (6 * rows * N if case["gated"] else 0), "flops": 20 * n}
    D = case["D"]
    n = B * S * D
    cols = 1 + (2 * rows if case["mod"] else 0)
    if op == "norm":
        return {"bytes": n * (6 if case["update"] else 2) + shown(n) + 2 * D * cols +
                (shown(n) + 4 * B * S if case["keep"] else 0), "flops": 10 * n}
    mod = rows if case["mod"] else 0
    return {"bytes": held(n) + 2 * n * (3 if case["stream"] else 2) + 2 * D * (1 + mod) +
            4 * D * (1 + 2 * mod) + 4 * B * S, "flops": 15 * n}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def _nearest(x):
    """x [..., K] in 64 bits as the blocks hold it: an exponent found by products, and codes rounded
    by their distance to the neighbours in their binade."""
    b = x.reshape(-1, 32)
    out = torch.empty_like(b)
    for i in range(0, b.shape[0], 1 << 20):
        c = b[i:i + (1 << 20)]
        top = c.abs().max(-1, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top)))) - 9.0
        e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e)
        e = torch.where(448.0 * torch.exp2(e) < top, e + 1, e)
        e = torch.where(top > 0, e, torch.full_like(e, -127.0)).clamp(min=-127.0)
        a = c / torch.exp2(e)
        # e4m3: three bits behind the leading one, down to 2^-6
        low = torch.log2(a.abs().clamp(min=2.0 ** -6)).floor()
        low = torch.where(torch.exp2(low) > a.abs().clamp(min=2.0 ** -6), low - 1, low)
        unit = torch.exp2(low - 3.0)
        out[i:i + (1 << 20)] = torch.round(a / unit) * unit * torch.exp2(e)
    return out.view(x.shape)


def _exact_matrix(codes, scales):
    """8-bit rows [..., K] as a matrix of 64 bits."""
    K = codes.shape[-1]
    bits = codes.reshape(-1, K).view(torch.uint8).long()
    E, m = bits % 128 // 8, bits % 8
    v = torch.where(E == 0, m * 2.0 ** -9, (1.0 + m.double() / 8.0) * torch.exp2(E.double() - 7.0))
    v = torch.where(bits >= 128, -v, v)
    r = torch.arange(v.shape[0], device=codes.device)[:, None]
    k = torch.arange(K // 32, device=codes.device)[None]
    byte = scales[((r // 128) * (-(-K // 128)) + k // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 +
                  k % 4]
    return v * torch.exp2(byte.double() - 127.0).repeat_interleave(32, dim=1)


def _act64(name, z):
    if name == "none":
        return z, torch.ones_like(z)
    if name == "silu":
        h = torch.nn.functional.silu(z)
    else:
        h = torch.nn.functional.gelu(z, approximate="tanh" if name == "gelu_tanh" else "none")
    # the derivative from a recorded pass
    with torch.enable_grad():
        v = z.detach().requires_grad_()
        y = torch.nn.functional.silu(v) if name == "silu" else torch.nn.functional.gelu(
            v, approximate="tanh" if name == "gelu_tanh" else "none")
        slope, = torch.autograd.grad(y.sum(), v)
    return h, slope


def _rows64(t, B, fill):
    """Modulation rows as [B, 1, D] in 64 bits; `fill` where there are none."""
    return fill if t is None else t.double().reshape(-1, 1, t.shape[-1]).expand(B, 1, -1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "weight_grad":
        def across(codes, scales):
            v = _exact_matrix(codes, scales)
            wide = torch.zeros(v.shape[1], -(-v.shape[0] // 32) * 32, dtype=torch.float64,
                               device="cuda")
            wide[:, :v.shape[0]] = v.t()
            return _nearest(wide)

        g = torch.einsum("nt,kt->nk", across(s["grad_z"], s["grad_z_scales"]),
                         across(s["x"], s["x_scales"]))
        return g if s["grad"] is None else g.add_(s["grad"])
    B, S = case["B"], case["S"]
    if op == "linear":
        N, K = case["N"], case["K"]
        x = _exact_matrix(s["x"], s["x_scales"]) if case["x8"] else \
            _nearest(s["x"].double().view(B * S, K))
        z = torch.matmul(x, _exact_matrix(s["w"], s["w_scales"]).t()).view(B, S, N)
        if case["bias"]:
            z += s["bias"].double()
        got = {"kept": _nearest(z)} if case["keep"] else {}
        y = _act64(case["act"], z)[0]
        if case["joined"]:
            y = torch.addcmul(s["residual"].double(), s["gate"].double(), y)
        got["out"] = _nearest(y) if case["quantize"] else y
        return got

    def fold(t):
        t = torch.einsum("bsd->bd", t)
        return t if case["per_batch"] else t.sum(0, keepdim=True)

    if op == "act_grad":
        N = case["N"]
        z = _exact_matrix(s["z"], s["z_scales"]).view(B, S, N)
        h, slope = _act64(case["act"], z)
        g = s["grad_out"].double()
        one = torch.ones(1, 1, N, dtype=torch.float64, device="cuda")
        dz = slope * g * _rows64(s["gate"], B, one)
        got = {"grad_z": _nearest(dz), "grad_bias": torch.einsum("bsd->d", dz)}
        if case["gated"]:
            got["grad_gate"] = fold(g * h)
        return got
    D = case["D"]
    one = torch.ones(1, 1, D, dtype=torch.float64, device="cuda")
    scale1 = 1.0 + _rows64(s["scale"], B, 0.0 * one)
    w = s["weight"].double() * one
    if op == "norm":
        T = s["x"].dtype
        res = s["x"].double()
        got = {}
        if case["update"]:
            got["res"] = res = res + s["update"].double()
        h = res.to(T).double()
        r = (torch.einsum("bsd,bsd->bs", h, h) / D + _EPS).rsqrt()
        got["out"] = _nearest(w * scale1 * h * r[..., None] +
                              _rows64(s["shift"], B, 0.0 * one))
        if case["keep"]:
            got["kept"], got["rstd"] = _nearest(h), r.view(-1)
        return got
    h = _exact_matrix(s["kept"], s["kept_scales"]).view(B, S, D)
    r = s["rstd"].double().view(B, S, 1)
    go = s["grad_out"].double()
    g = go * (w * scale1)
    dx = g * r - h * (r ** 3) * (torch.einsum("bsd,bsd->bs", g, h)[..., None] / D)
    if s["grad_res"] is not None:
        dx += s["grad_res"].double()
    p = go * h * r
    got = {"grad_x": dx, "grad_weight": torch.einsum("bsd->d", p * scale1)}
    if case["mod"]:
        got["grad_scale"], got["grad_shift"] = fold(p * w), fold(go)
    return got
