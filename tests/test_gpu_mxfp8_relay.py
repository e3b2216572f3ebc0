"""The 8-bit operators one after the other on the same buffers: each launch reads what the one before it
has just written, and the next round writes it anew while kernels that were launched early wait.  The
results are those of the same calls on buffers of their own, with the device waited for after each."""
import pytest
import torch

pytestmark = pytest.mark.gpu

ROUNDS = 12


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


class Relay:
    """Buffers of one round's intermediate results, or none: then every call allocates."""

    def __init__(self, rm, B, S, D, own):
        self.rm, self.B, self.S, self.D, self.own = rm, B, S, D, own
        e = lambda *s, t=torch.bfloat16: torch.empty(*s, device="cuda", dtype=t)  # noqa: E731
        new = lambda *s: rm.Mxfp8(  # noqa: E731
            e(*s, t=torch.float8_e4m3fn),
            e(rm.mxfp8_scale_bytes(e(*s).numel() // s[-1], s[-1]), t=torch.uint8))
        R = -(-B * S // 32) * 32
        self.buf = dict(mod=e(B, 3 * D), res=e(B, S, D), h=new(B, S, D), kept=new(B, S, D),
                        y=new(B, S, D), z=new(B, S, D), dz=new(B, S, D), turned=new(D, R),
                        flat=e(D, R)) if own else {}
        self.work = [e(n, t=torch.uint8) for n in (
            rm.library().mxfp8_activation_backward_workspace_bytes(B, S, D),
            rm.library().rmsnorm_mxfp8_backward_workspace_bytes(B, S, D))] if own else [None, None]

    def round(self, t, w, wm, after=lambda: None):
        rm, g = self.rm, self.buf.get

        def done(v):
            after()
            return v

        # the row vectors are a product's results too
        mod = done(rm.mxfp8_linear(t["c"], wm, out=g("mod")))
        scale, shift, gate = mod.view(self.B, 1, -1).chunk(3, -1)
        rstd = torch.empty(self.B * self.S, device="cuda")
        res, h, kept = done(rm.add_rmsnorm_mxfp8(t["x"], t["u"], None, scale, shift, keep=g("kept") or True,
                                                 res_out=g("res"), out=g("h"), rstd_out=rstd))
        y, z = done(rm.mxfp8_linear(h, w, activation="silu", gate=gate, residual=res, out=g("y"),
                                    quantize=True, keep=g("z") or True))
        dz, db, dgate = done(rm.mxfp8_activation_backward(z, res, "silu", gate, out=g("dz"),
                                                          workspace=self.work[0]))
        turned = done(rm.mxfp8_transpose(dz, out=g("turned")))
        flat = done(rm.mxfp8_dequantize(turned, out=g("flat")))
        grads = done(rm.rmsnorm_mxfp8_backward(kept, None, scale, res, rstd, workspace=self.work[1]))
        seen = [flat, rm.mxfp8_dequantize(y), db, dgate, grads[0], *grads[2:]]
        return [v.clone() for v in seen]


@pytest.mark.parametrize("B,S,D", [(3, 1, 128), (2, 77, 512), (4, 300, 2080), (1, 1000, 4096)])
@pytest.mark.parametrize("graph", [False, True])
def test_rounds_on_the_same_buffers(rm, B, S, D, graph):
    gen = torch.Generator(device="cuda").manual_seed(B + S + D)
    n = lambda *s: torch.randn(*s, device="cuda", generator=gen).bfloat16()  # noqa: E731
    w, wm = rm.mxfp8_quantize(n(D, D) * D ** -0.5), rm.mxfp8_quantize(n(3 * D, D) * D ** -0.5)
    given = [dict(c=n(B, D), x=n(B, S, D) * 2.0 ** (i % 5), u=n(B, S, D)) for i in range(ROUNDS)]
    alone = Relay(rm, B, S, D, own=False)
    want = [alone.round(t, w, wm, after=torch.cuda.synchronize) for t in given]
    same = Relay(rm, B, S, D, own=True)
    run = lambda: [same.round(t, w, wm) for t in given]  # noqa: E731
    if graph:
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        for _ in range(3):
            g.replay()
    else:
        got = run()
    for a, b in zip(got, want):
        for p, q in zip(a, b):
            assert torch.equal(p, q)
