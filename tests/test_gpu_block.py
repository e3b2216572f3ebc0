"""The sandwich norms and the 4-bit projections together, as a block uses them: two blocks forward,
each stage against float64 on the values that the stage before left; two blocks backward against
float64 autograd; the same from a replayed graph and from several streams at once."""
import pytest
import torch

import _sandwich as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
B, S, D, H = 2, 150, 512, 1536


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


class Block:
    def __init__(self, rm, gen):
        n = lambda *s: torch.randn(*s, device="cuda", generator=gen)  # noqa: E731
        self.pre, self.post = ((1 + 0.05 * n(D)).bfloat16() for _ in range(2))
        self.gate, self.scale, self.shift = (0.3 * n(B, 1, 3 * D)).bfloat16().chunk(3, -1)
        self.up = rm.mxfp4_quantize((n(H, D) / D ** 0.5).bfloat16())
        self.down = rm.mxfp4_quantize((n(D, H) / H ** 0.5).bfloat16())
        self.bias = (0.1 * n(H)).bfloat16()


def forward(rm, blocks, stream, update):
    """-> every stage's result: the stream joins an update, is normalised for the block, and the
    block's two projections make the next update."""
    seen = []
    for b in blocks:
        res, out = rm.sandwich_rmsnorm_modulate(stream, update, b.post, b.gate, b.pre, b.scale,
                                                b.shift)
        mid = rm.mxfp4_linear(out, b.up, bias=b.bias)
        update = rm.mxfp4_linear(mid, b.down)
        seen.append((stream, res, out, mid, update))
        stream = res
    # the last block ends without a norm of its own: gate and residual in the product
    b = blocks[-1]
    last = rm.mxfp4_linear(seen[-1][3], b.down, gate=b.gate, residual=stream)
    return seen, last


def near(got, want, size, steps):
    bound = 2.0 ** -8 * want.abs() + steps * U * size + 1e-30
    off = ((got.double() - want).abs() / bound).max().item()
    assert off <= 1.0, off


def linear64(rm, x, w):
    a, b = (rm.mxfp4_dequantize(q).double() for q in (rm.mxfp4_quantize(x), w))
    return a @ b.T, a.abs() @ b.abs().T


def make(rm, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [Block(rm, gen) for _ in range(2)]
    stream, update = (torch.randn(B, S, D, device="cuda", generator=gen).bfloat16()
                      for _ in range(2))
    return blocks, stream, update


def test_two_blocks_forward(rm):
    blocks, stream, update = make(rm)
    seen, last = forward(rm, blocks, stream, update)
    for b, (stream, res, out, mid, made) in zip(blocks, seen):
        near(res, *ref.residual_add(stream, update, b.post, b.gate, 1e-6, 1.0, 1.0), 64)
        near(out, *ref.norm(res, b.pre, b.scale, b.shift, 1e-6), 64)
        # a product's step of 64 values adds with an error of 2^-23 of the magnitudes at most
        want, size = linear64(rm, out, b.up)
        near(mid, want + b.bias.double(), size + b.bias.double().abs(), 2 * (D / 64 + 4))
        want, size = linear64(rm, mid, b.down)
        near(made, want, size, 2 * (H / 64 + 4))
        update = made
    b = blocks[-1]
    g = b.gate.double()
    near(last, seen[-1][1].double() + g * want, seen[-1][1].double().abs() + g.abs() * size,
         2 * (H / 64 + 4))


def test_two_blocks_from_a_graph_and_from_streams(rm):
    blocks, stream, update = make(rm, 1)
    want = forward(rm, blocks, stream, update)[1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = forward(rm, blocks, stream, update)[1]
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    # many rows and few rows at once, on four streams
    few = [t[:, :3].contiguous() for t in (stream, update)]
    want_few = forward(rm, blocks, *few)[1]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    results = []
    for i in range(12):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                args = few if (i + k) % 2 else (stream, update)
                results.append(((i + k) % 2, forward(rm, blocks, *args)[1]))
    torch.cuda.synchronize()
    for is_few, r in results:
        assert torch.equal(r, want_few if is_few else want)


def test_two_sandwiches_backward(rm):
    """The gradient of a loss over two sandwich norms in a row, against autograd in float64 with the
    stored values in their places (the roundings pass gradients straight through)."""
    blocks, stream, update = make(rm, 2)
    gen = torch.Generator(device="cuda").manual_seed(9)
    updates = [update, torch.randn(B, S, D, device="cuda", generator=gen).bfloat16()]
    weight = [torch.randn(B, S, D, device="cuda", generator=gen).bfloat16() for _ in range(3)]
    kept, x = [], stream
    for b, u in zip(blocks, updates):
        rp, r = (torch.empty(B * S, dtype=torch.float32, device="cuda") for _ in range(2))
        res, out = rm.sandwich_rmsnorm_modulate(x, u, b.post, b.gate, b.pre, b.scale, b.shift,
                                                post_rstd_out=rp, rstd_out=r)
        kept.append((x, res, rp, r))
        x = res
    # loss = <out0, w0> + <out1, w1> + <res1, w2>
    grads, flow = [None, None], weight[2]
    for i in (1, 0):
        b = blocks[i]
        _, res, rp, r = kept[i]
        grads[i] = rm.sandwich_rmsnorm_modulate_backward(updates[i], res, b.post, b.gate, b.pre,
                                                         b.scale, flow, weight[i], rp, r)
        flow = grads[i].residual
    d = lambda t: t.double().detach().requires_grad_()  # noqa: E731
    leaves = [dict(update=d(u), post_weight=d(b.post), gate=d(b.gate), weight=d(b.pre),
                   scale=d(b.scale), shift=d(b.shift)) for b, u in zip(blocks, updates)]
    first = d(stream)
    x, loss = first, 0.0
    for leaf, (_, res, _, _), w in zip(leaves, kept, weight):
        v = leaf["update"] * (leaf["update"].square().mean(-1, keepdim=True) + 1e-6).rsqrt()
        y = x + v * leaf["post_weight"] * leaf["gate"]
        x = y + (res.double() - y).detach()  # as stored
        o = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * leaf["weight"]
        loss = loss + ((o * (1 + leaf["scale"]) + leaf["shift"]) * w.double()).sum()
    (loss + (x * weight[2].double()).sum()).backward()
    # the second block's stored gradient is off by half a step of each of its values, 2^-8, and
    # passes through the first block's norms, whose Jacobians (of unit-size rows) stretch no vector;
    # 2^-8 of each value again for the stored result.  In the 2-norm over a tensor:
    for i, leaf in enumerate(leaves):
        for name, p in leaf.items():
            got = getattr(grads[i], name).double().view(p.shape)
            off = (got - p.grad).norm() / p.grad.norm()
            assert off <= 2 * 2.0 ** -8, (i, name, off.item())
    off = (grads[0].residual.double() - first.grad).norm() / first.grad.norm()
    assert off <= 2 * 2.0 ** -8
