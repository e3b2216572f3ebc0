"""Workspaces of the 8-bit gradients: as large as the call's own form asks for (row vectors of every batch
or of all), whether the call allocates them or the caller does, and what lies behind them is not touched."""
import pytest
import torch

pytestmark = pytest.mark.gpu

# calls whose form is the other one than the largest of their sizes
SHAPES = [(300, 1, 512), (40, 3, 2080), (3, 200, 1024)]


@pytest.fixture(scope="module")
def rm():
    import rmsnorm_modulate_gb300 as rm

    yield rm
    assert rm.device_status(clear=True) == 0


def n(*s):
    return torch.randn(*s, device="cuda").bfloat16()


def act(rm, B, S, N, rows):
    z = rm.mxfp8_quantize(n(B, S, N))
    g, gate = n(B, S, N), None if rows is None else n(rows, 1, N)
    return lambda w=None: rm.mxfp8_activation_backward(z, g, "silu", gate, workspace=w)


def norm(rm, B, S, D, rows):
    kept = rm.mxfp8_quantize(n(B, S, D))
    go, scale = n(B, S, D), None if rows is None else n(rows, 1, D)
    weight, rstd = n(D), torch.rand(B * S, device="cuda") + 0.5
    return lambda w=None: rm.rmsnorm_mxfp8_backward(kept, weight, scale, go, rstd, workspace=w)


def tensors(v):
    return [t for u in v for t in tensors(u)] if isinstance(v, tuple) else [] if v is None else [v]


@pytest.mark.parametrize("call,name", [(act, "mxfp8_activation_backward"),
                                       (norm, "rmsnorm_mxfp8_backward")])
@pytest.mark.parametrize("form", ["batch", "one", None])
@pytest.mark.parametrize("B,S,D", SHAPES)
def test_workspace_of_the_form(rm, B, S, D, form, call, name):
    run = call(rm, B, S, D, {"batch": B, "one": 1, None: None}[form])
    need = getattr(rm.library(), name + "_workspace_bytes")(*((B, S) if form == "batch" else (1, B * S)), D)
    want = run()
    area = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    got = run(area[:need])
    for a, b in zip(tensors(want), tensors(got)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert (area[need:] == 0xA5).all()
    with pytest.raises(ValueError):
        run(area[:need - 1])


@pytest.mark.parametrize("call", [act, norm])
@pytest.mark.parametrize("form", [1, None])
def test_many_batches_under_one_row_allocate_little(rm, call, form):
    run = call(rm, 4096, 1, 4096, form)
    made = sum(t.numel() * t.element_size() for t in tensors(run()))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    run()
    # a run or a piece is 27 rows or more, and leaves two rows of fp32
    assert torch.cuda.max_memory_allocated() - before - made <= 4096 // 27 * 2 * 4096 * 4 + (1 << 20)
