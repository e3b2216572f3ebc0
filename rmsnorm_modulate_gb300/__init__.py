"""rmsnorm_modulate_gb300 -- fused adaLN row normalisation + modulate for GB300.

Thin ctypes binding of ``librmsmod.so`` (C ABI in ``include/rmsmod.h``).
Each function here only checks tensor metadata, derives sizes and strides,
and passes device pointers plus the current CUDA stream to the library;
every step of the computation runs in the library's CUDA kernels.  There is
no CPU fallback: if the library is not built, or the tensors are not on a
CUDA device, the call raises.

Tensors are ``torch.bfloat16`` on a CUDA device with a contiguous innermost
dimension (the sandwich norms, the 4-bit and the 8-bit calls take ``torch.float16`` too,
and run on their tensors' device whichever is current).  Modulation rows (``scale``, ``shift``, ``gate``) may be given
as ``[D]``, ``[1, D]``, ``[B, D]``, ``[1, 1, D]`` or ``[B, 1, D]``; per-batch
rows may be strided views (adaLN chunk views of one projection output).

Every call takes a ``stream`` (default: the current one), which the caller orders after its inputs.
What the sandwich norms, rmsnorm_modulate_backward, the 4-bit and the 8-bit calls allocate is that stream's, and
the current stream is noted as using their results; the other calls allocate on the current stream,
so with another one pass them their outputs.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
import threading
from typing import NamedTuple

import torch

__all__ = [
    "RmsmodError", "library", "library_path", "ln_modulate", "ln_modulate_folded",
    "ln_modulate_backward", "ln_modulate_backward_static", "backward_workspace_bytes",
    "rmsnorm_modulate",
    "gated_rmsnorm_modulate", "qk_layernorm", "rmsnorm_silu_cl", "modulate_scale_shift",
    "residual_gate_add", "conv_bias_epilogue", "sandwich_rmsnorm_modulate",
    "sandwich_rmsnorm_modulate_backward", "SandwichGrads", "rmsnorm_modulate_backward", "Mxfp4", "mxfp4_quantize", "mxfp4_dequantize",
    "mxfp4_scale_bytes", "mxfp4_linear", "Mxfp8", "mxfp8_scale_bytes", "mxfp8_quantize",
    "mxfp8_dequantize", "mxfp8_transpose", "mxfp8_linear", "mxfp8_activation_backward",
    "add_rmsnorm_mxfp8", "rmsnorm_mxfp8_backward", "supported", "status_string", "device_status",
    "selftest_wait_timeout",
    "OP_LN_MODULATE", "OP_RMSNORM_MODULATE", "OP_GATED_RMSNORM_MODULATE",
    "OP_QK_LAYERNORM", "OP_RMSNORM_SILU_CL", "OP_LN_MODULATE_FOLDED",
    "OP_SANDWICH_RMSNORM_MODULATE", "OP_MXFP4", "OP_MXFP8", "OP_ADD_RMSNORM_MXFP8",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "librmsmod.so")

OP_LN_MODULATE = 1
OP_RMSNORM_MODULATE = 2
OP_GATED_RMSNORM_MODULATE = 3
OP_QK_LAYERNORM = 4
OP_RMSNORM_SILU_CL = 5
OP_LN_MODULATE_FOLDED = 6
OP_SANDWICH_RMSNORM_MODULATE = 7
OP_MXFP4 = 8
OP_MXFP8 = 9
OP_ADD_RMSNORM_MXFP8 = 10

_lock = threading.Lock()
_lib = None


class RmsmodError(RuntimeError):
    """A non-zero status returned by librmsmod."""

    def __init__(self, status: int, func: str):
        self.status = status
        super().__init__(f"{func}: status {status}: {status_string(status)}")


def library_path() -> str:
    return _LIB_PATH


def library() -> ctypes.CDLL:
    """The loaded librmsmod.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is not built: run `python -m rmsnorm_modulate_gb300._build` "
                "or __graft_entry__.build()")
        lib = ctypes.CDLL(_LIB_PATH)
        P, I, F, C = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_int
        sig = {
            "ln_modulate": [P, P, P, P, I, I, I, I, F, P, P, P],
            "ln_modulate_folded": [P, P, P, P, I, I, I, I, F, P, P, P],
            "modulate_scale_shift_f16": [P, P, P, P, I, I, I, I, P],
            "ln_modulate_backward": [P, P, I, P, P, P, I, I, I, P, P, P, P, ctypes.c_size_t, P],
            "ln_modulate_backward_static": [P, P, I, P, P, P, I, I, I, P, P, P, P],
            "rmsnorm_modulate": [P, P, P, P, P, I, I, I, I, F, P, P],
            "gated_rmsnorm_modulate": [P, P, P, I, P, P, P, I, P, P, I, I, I, F, P, P],
            "qk_layernorm": [P, P, P, P, P, P, P, P, I, I, I, F, P, P, P],
            "qk_layernorm_strided": [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, I, F, P, P, P],
            "rmsnorm_silu_cl": [P, P, C, P, P, I, I, F, P, P],
            "modulate_scale_shift": [P, P, P, P, I, I, I, I, P],
            "residual_gate_add": [P, P, P, I, P, I, I, I, P],
            "conv_bias_epilogue": [P, P, C, P, P, I, I, P],
            "sandwich_rmsnorm_modulate": [P, P, P, P, I, P, P, P, I, P, P, I, I, I, F, F, F, F, P,
                                          P, C, P],
            "sandwich_rmsnorm_modulate_backward": [P, P, P, P, I, P, P, I, P, P, P, P, I, I, I, F,
                                                   F, P, P, P, P, P, P, P, P, ctypes.c_size_t, C,
                                                   P],
            "rmsnorm_modulate_backward": [P, P, P, I, P, P, P, I, I, I, P, P, P, P, P,
                                          ctypes.c_size_t, P],
            "mxfp4_quantize": [P, P, P, I, I, C, P],
            "mxfp4_dequantize": [P, P, P, I, I, C, P],
            "mxfp4_matmul": [P, P, P, P, P, P, I, P, P, I, I, I, I, C, P],
            "mxfp8_quantize": [P, P, P, I, I, C, P],
            "mxfp8_dequantize": [P, P, P, I, I, C, P],
            "mxfp8_transpose": [P, P, P, P, I, I, P],
            "mxfp8_matmul": [P, P, P, P, P, C, P, I, P, P, P, P, P, I, I, I, I, C, P],
            "mxfp8_activation_backward": [P, P, P, C, P, I, P, P, P, P, I, I, I, P,
                                          ctypes.c_size_t, C, P],
            "add_rmsnorm_mxfp8": [P, P, P, P, P, I, P, P, P, P, P, I, I, I, F, P, C, P],
            "rmsnorm_mxfp8_backward": [P, P, P, P, I, P, P, P, I, I, I, P, P, P, P, P,
                                       ctypes.c_size_t, C, P],
            "rmsmod_supported": [C, I, ctypes.POINTER(P), C],
            "rmsmod_status_string": [C],
            "rmsmod_version": [],
            "rmsmod_device_status": [ctypes.POINTER(ctypes.c_uint), C],
            "rmsmod_selftest_wait_timeout": [ctypes.c_uint64, P],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.rmsmod_status_string.restype = ctypes.c_char_p
        for name in ("sandwich_rmsnorm_modulate_backward_workspace_bytes",
                     "rmsnorm_modulate_backward_workspace_bytes",
                     "rmsnorm_mxfp8_backward_workspace_bytes",
                     "mxfp8_activation_backward_workspace_bytes"):
            getattr(lib, name).argtypes = [I, I, I]
            getattr(lib, name).restype = ctypes.c_size_t
        for name in ("mxfp4_scale_bytes", "mxfp8_scale_bytes"):
            getattr(lib, name).argtypes = [I, I]
            getattr(lib, name).restype = ctypes.c_size_t
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return library().rmsmod_status_string(int(status)).decode()


def _call(name: str, *args) -> None:
    st = getattr(library(), name)(*args)
    if st != 0:
        raise RmsmodError(st, name)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


_entries = {}  # the library's functions by name, once looked up

# (torch without CUDA has neither, and no call gets that far)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _entry(name):
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(library(), name)
    return fn


def _call_on(device, stream, name, *args) -> None:
    """Call `name` on the tensors' own device, with `stream` (None: that device's current one) as the
    last argument.  Pointers are passed as integers (_at): half of a small call's time would
    otherwise go into ctypes objects."""
    index = device.index
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    fn = _entries.get(name) or _entry(name)
    if index == _current_device():
        st = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            st = fn(*args, raw)
    if st:
        raise RmsmodError(st, name)


def _at(t):
    return None if t is None else t.data_ptr()


def _aside(stream, device, call, *args):
    """call(*args, None), a call whose last argument is its stream, with `stream` as the current one.
    For calls that allocate: the memory comes from that stream's own pool, so that nothing on another
    stream can be given it while the call's work still writes it, and the results are noted as used by
    the caller's current stream, so that it is not taken again before what that one does is done.
    (On the host that takes some 20 us, which a call that is given its results does without.)"""
    if stream.device != device:
        raise ValueError(f"stream must be on {device}")
    current = torch.cuda.current_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return call(*args, None)
    with torch.cuda.stream(stream):
        made = call(*args, None)
    _shared_with(made, current)
    return made


def _shared_with(made, stream):
    """Note `stream` on a call's results, however they are grouped."""
    if isinstance(made, tuple):
        for t in made:
            _shared_with(t, stream)
    elif made is not None:
        made.record_stream(stream)


def _bf16(t, name, dtype=torch.bfloat16):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    return t


def _dense(t, name, dtype=torch.bfloat16):
    _bf16(t, name, dtype)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _f32_out(t, n, name, device):
    if t is None:
        return None
    if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of {n} elements")
    return t


def _mod_rows(t, B, D, name, dtype=torch.bfloat16):
    """-> batch stride in elements (0 = one row shared by every batch)."""
    _bf16(t, name, dtype)
    if t.shape[-1] != D or t.stride(-1) != 1:
        raise ValueError(f"{name} must end in a unit-stride dimension of size {D}")
    rows = t.numel() // D if D else math.prod(t.shape[:-1])
    if rows == 1:
        return 0
    if rows != B:
        raise ValueError(f"{name} has {rows} rows, expected 1 or B={B}")
    # the one non-trivial leading dimension carries the batch stride
    for size, stride in zip(t.shape[:-1], t.stride()[:-1]):
        if size == B:
            return stride
    raise ValueError(f"{name}: cannot find the batch dimension")


def _bsd(x, name="x", dtype=torch.bfloat16):
    _dense(x, name, dtype)
    if x.dim() == 2:
        return 1, x.shape[0], x.shape[1]
    if x.dim() != 3:
        raise ValueError(f"{name} must be [B, S, D] or [S, D]")
    return x.shape[0], x.shape[1], x.shape[2]


def _out_like(out, x, name="out"):
    if out is None:
        return torch.empty_like(x)
    _dense(out, name, x.dtype)
    if out.shape != x.shape:
        raise ValueError(f"{name} shape {tuple(out.shape)} != {tuple(x.shape)}")
    return out


def ln_modulate(x, scale, shift, eps: float = 1e-6, out=None, mean_out=None, rstd_out=None,
                stream=None):
    """LayerNorm (no affine) over the last dim, then R(R(y * R(1 + scale)) + shift)."""
    B, S, D = _bsd(x)
    bs = _mod_rows(scale, B, D, "scale")
    if _mod_rows(shift, B, D, "shift") != bs:
        raise ValueError("scale and shift must share one batch stride")
    out = _out_like(out, x)
    _f32_out(mean_out, B * S, "mean_out", x.device)
    _f32_out(rstd_out, B * S, "rstd_out", x.device)
    _call("ln_modulate", _ptr(x), _ptr(scale), _ptr(shift), _ptr(out), B, S, D, bs, eps,
          _ptr(mean_out), _ptr(rstd_out), _stream(stream))
    return out


def ln_modulate_folded(x, scale, shift, eps: float = 1e-6, out=None, mean_out=None,
                       rstd_out=None, stream=None):
    """Single-rounding tier: R(((x - mean) * rstd) * R(1 + scale) + shift) (not bit-exact
    with the eager chain; same arguments as ln_modulate)."""
    B, S, D = _bsd(x)
    bs = _mod_rows(scale, B, D, "scale")
    if _mod_rows(shift, B, D, "shift") != bs:
        raise ValueError("scale and shift must share one batch stride")
    out = _out_like(out, x)
    _f32_out(mean_out, B * S, "mean_out", x.device)
    _f32_out(rstd_out, B * S, "rstd_out", x.device)
    _call("ln_modulate_folded", _ptr(x), _ptr(scale), _ptr(shift), _ptr(out), B, S, D, bs, eps,
          _ptr(mean_out), _ptr(rstd_out), _stream(stream))
    return out


def backward_workspace_bytes(B: int, S: int, D: int) -> int:
    """Device workspace ln_modulate_backward needs for the token sums."""
    lib = library()
    f = lib.ln_modulate_backward_workspace_bytes
    f.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]
    f.restype = ctypes.c_size_t
    return int(f(B, S, D))


def ln_modulate_backward(x, scale, grad_out, mean, rstd, need_x=True, need_mod=True,
                         grad_x=None, grad_scale=None, grad_shift=None, workspace=None,
                         stream=None):
    """Gradients of ln_modulate (x, scale rows as in the forward; mean, rstd the
    forward's fp32 statistics).  -> (grad_x bf16 like x or None, grad_scale fp32
    [B, D] or None, grad_shift fp32 [B, D] or None).  grad_scale / grad_shift
    are batch-invariant token sums (fixed 32-way trees); the workspace they need
    is allocated here unless one is passed."""
    B, S, D = _bsd(x)
    bs = _mod_rows(scale, B, D, "scale")
    _dense(grad_out, "grad_out")
    if grad_out.shape != x.shape:
        raise ValueError("grad_out must match x")
    _f32_out(mean, B * S, "mean", x.device)
    _f32_out(rstd, B * S, "rstd", x.device)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd (the forward's statistics) are required")
    if need_x:
        grad_x = _out_like(grad_x, x, "grad_x")
    else:
        grad_x = None
    if need_mod:
        if grad_scale is None:
            grad_scale = torch.empty(B, D, dtype=torch.float32, device=x.device)
        if grad_shift is None:
            grad_shift = torch.empty(B, D, dtype=torch.float32, device=x.device)
        _f32_out(grad_scale, B * D, "grad_scale", x.device)
        _f32_out(grad_shift, B * D, "grad_shift", x.device)
        need = backward_workspace_bytes(B, S, D)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
        elif workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace holds fewer than the {need} bytes needed")
        wbytes = workspace.numel() * workspace.element_size()
    else:
        grad_scale = grad_shift = None
        workspace, wbytes = None, 0
    _call("ln_modulate_backward", _ptr(x), _ptr(scale), bs, _ptr(grad_out), _ptr(mean),
          _ptr(rstd), B, S, D, _ptr(grad_x), _ptr(grad_scale), _ptr(grad_shift),
          _ptr(workspace), wbytes, _stream(stream))
    return grad_x, grad_scale, grad_shift


def ln_modulate_backward_static(x, scale, grad_out, mean, rstd, grad_x, grad_scale,
                                grad_shift, stream=None):
    """ln_modulate_backward through the entry point that uses the library's
    fixed 8 MiB device scratch instead of a workspace (allocates nothing; every
    output is passed in, None to skip it).  Calls overlapping in time race."""
    B, S, D = _bsd(x)
    bs = _mod_rows(scale, B, D, "scale")
    _dense(grad_out, "grad_out")
    if grad_out.shape != x.shape:
        raise ValueError("grad_out must match x")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd (the forward's statistics) are required")
    _f32_out(mean, B * S, "mean", x.device)
    _f32_out(rstd, B * S, "rstd", x.device)
    if grad_x is not None:
        _out_like(grad_x, x, "grad_x")
    _f32_out(grad_scale, B * D, "grad_scale", x.device)
    _f32_out(grad_shift, B * D, "grad_shift", x.device)
    _call("ln_modulate_backward_static", _ptr(x), _ptr(scale), bs, _ptr(grad_out), _ptr(mean),
          _ptr(rstd), B, S, D, _ptr(grad_x), _ptr(grad_scale), _ptr(grad_shift),
          _stream(stream))
    return grad_x, grad_scale, grad_shift


def rmsnorm_modulate(x, weight, scale, shift, eps: float = 1e-6, out=None, rstd_out=None,
                     stream=None):
    """RMSNorm (weight may be None) over the last dim, then the modulate chain."""
    B, S, D = _bsd(x)
    if weight is not None:
        _dense(weight, "weight")
        if weight.numel() != D:
            raise ValueError("weight must have D elements")
    bs = _mod_rows(scale, B, D, "scale")
    if _mod_rows(shift, B, D, "shift") != bs:
        raise ValueError("scale and shift must share one batch stride")
    out = _out_like(out, x)
    _f32_out(rstd_out, B * S, "rstd_out", x.device)
    _call("rmsnorm_modulate", _ptr(x), _ptr(weight), _ptr(scale), _ptr(shift), _ptr(out), B, S,
          D, bs, eps, _ptr(rstd_out), _stream(stream))
    return out


def gated_rmsnorm_modulate(residual, update, gate, weight, scale, shift, eps: float = 1e-6,
                           res_out=None, out=None, rstd_out=None, stream=None):
    """res = R(residual + R(gate * update)); out = rmsnorm_modulate(res).  -> (res, out)."""
    B, S, D = _bsd(residual, "residual")
    _dense(update, "update")
    if update.shape != residual.shape:
        raise ValueError("update must match residual")
    gs = _mod_rows(gate, B, D, "gate")
    if weight is not None:
        _dense(weight, "weight")
        if weight.numel() != D:
            raise ValueError("weight must have D elements")
    bs = _mod_rows(scale, B, D, "scale")
    if _mod_rows(shift, B, D, "shift") != bs:
        raise ValueError("scale and shift must share one batch stride")
    res_out = _out_like(res_out, residual, "res_out")
    out = _out_like(out, residual)
    _f32_out(rstd_out, B * S, "rstd_out", residual.device)
    _call("gated_rmsnorm_modulate", _ptr(residual), _ptr(update), _ptr(gate), gs, _ptr(weight),
          _ptr(scale), _ptr(shift), bs, _ptr(res_out), _ptr(out), B, S, D, eps, _ptr(rstd_out),
          _stream(stream))
    return res_out, out


def _token_view(t, name):
    """[..., heads, head_dim] view with dense heads and one uniform stride
    over the leading dims -> (tokens, heads, token_stride in elements)."""
    _bf16(t, name)
    if t.dim() < 2 or t.stride(-1) != 1 or (t.dim() >= 2 and t.shape[-2] > 1 and
                                             t.stride(-2) != t.shape[-1]):
        raise ValueError(f"{name}: heads must be dense [..., heads, head_dim]")
    heads, hd = (t.shape[-2], t.shape[-1]) if t.dim() >= 2 else (1, t.shape[-1])
    lead = list(zip(t.shape[:-2], t.stride()[:-2]))
    tokens, ts = 1, heads * hd
    for size, stride in reversed(lead):
        if size == 1:
            continue
        if tokens == 1:
            ts = stride
        elif stride != ts * tokens:
            raise ValueError(f"{name}: leading dims do not collapse to one token stride")
        tokens *= size
    return tokens, heads, ts


def qk_layernorm(q, k, wq, bq, wk, bk, eps: float = 1e-5, q_out=None, k_out=None,
                 mean_out=None, rstd_out=None, stream=None):
    """Per-head LayerNorm(head_dim) with affine on q and k in one launch. -> (q_out, k_out).
    q / k may be token-strided views (e.g. slices of a fused QKV projection)
    whose heads are dense; head_dim 64, 96 or 128."""
    hd = q.shape[-1]
    if k.shape[-1] != hd:
        raise ValueError("q and k must share head_dim")
    for t, n in ((wq, "wq"), (bq, "bq"), (wk, "wk"), (bk, "bk")):
        _dense(t, n)
        if t.numel() != hd:
            raise ValueError(f"{n} must have head_dim elements")
    dense = all(t.is_contiguous() for t in (q, k)) and all(
        t is None or t.is_contiguous() for t in (q_out, k_out))
    if dense:
        _dense(q, "q")
        _dense(k, "k")
        rq, rk = q.numel() // hd, k.numel() // hd
        q_out = _out_like(q_out, q, "q_out")
        k_out = _out_like(k_out, k, "k_out")
        _f32_out(mean_out, rq + rk, "mean_out", q.device)
        _f32_out(rstd_out, rq + rk, "rstd_out", q.device)
        _call("qk_layernorm", _ptr(q), _ptr(k), _ptr(wq), _ptr(bq), _ptr(wk), _ptr(bk),
              _ptr(q_out), _ptr(k_out), rq, rk, hd, eps, _ptr(mean_out), _ptr(rstd_out),
              _stream(stream))
        return q_out, k_out
    tq, hq, qts = _token_view(q, "q")
    tk, hk, kts = _token_view(k, "k")
    if tq != tk:
        raise ValueError("q and k must have the same number of tokens")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    if q_out.shape != q.shape or k_out.shape != k.shape:
        raise ValueError("q_out / k_out must match q / k")
    to, _, qots = _token_view(q_out, "q_out")
    _, _, kots = _token_view(k_out, "k_out")
    rows = tq * (hq + hk)
    _f32_out(mean_out, rows, "mean_out", q.device)
    _f32_out(rstd_out, rows, "rstd_out", q.device)
    _call("qk_layernorm_strided", _ptr(q), _ptr(k), _ptr(wq), _ptr(bq), _ptr(wk), _ptr(bk),
          _ptr(q_out), _ptr(k_out), tq, hq, hk, hd, qts, kts, qots, kots, eps, _ptr(mean_out),
          _ptr(rstd_out), _stream(stream))
    return q_out, k_out


def _pixels_c(x):
    """Dense channels-last activation -> (pixels, C).  Accepts [..., C] contiguous
    tensors or channels_last(_3d) N C (T) H W tensors."""
    if x.dim() in (4, 5) and not x.is_contiguous():
        fmt = torch.channels_last if x.dim() == 4 else torch.channels_last_3d
        if not x.is_contiguous(memory_format=fmt):
            raise ValueError("x must be dense channels-last")
        return x.numel() // x.shape[1], x.shape[1]
    if not x.is_contiguous():
        raise ValueError("x must be dense channels-last")
    if x.dim() in (4, 5):
        raise ValueError("a 4-D/5-D x must be in channels_last(_3d) memory format")
    return x.numel() // x.shape[-1], x.shape[-1]


def rmsnorm_silu_cl(x, bias, gamma, eps: float = 1e-6, out=None, rstd_out=None, stream=None):
    """SiLU(RMSNorm_C(x + bias) * gamma) on a channels-last activation."""
    _bf16(x, "x")
    pixels, C = _pixels_c(x)
    if bias is not None:
        if bias.dtype not in (torch.float32, torch.bfloat16) or not bias.is_cuda or \
                bias.numel() != C or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous fp32/bf16 CUDA tensor of C elements")
    _dense(gamma, "gamma")
    if gamma.numel() != C:
        raise ValueError("gamma must have C elements")
    if out is None:
        out = torch.empty_like(x)  # keeps the channels-last strides
    elif out.shape != x.shape or out.stride() != x.stride() or out.dtype != torch.bfloat16:
        raise ValueError("out must match x's shape, strides and dtype")
    _f32_out(rstd_out, pixels, "rstd_out", x.device)
    is32 = 1 if (bias is not None and bias.dtype == torch.float32) else 0
    _call("rmsnorm_silu_cl", _ptr(x), _ptr(bias), is32, _ptr(gamma), _ptr(out), pixels, C, eps,
          _ptr(rstd_out), _stream(stream))
    return out


def modulate_scale_shift(y, scale, shift, out=None, stream=None):
    """R(R(y * R(1 + scale)) + shift) over y [B, S, D], in y's storage type
    (bfloat16 or float16; scale and shift must match it)."""
    if isinstance(y, torch.Tensor) and y.dtype == torch.float16:
        dt, entry = torch.float16, "modulate_scale_shift_f16"
    else:
        dt, entry = torch.bfloat16, "modulate_scale_shift"
    B, S, D = _bsd(y, "y", dt)
    bs = _mod_rows(scale, B, D, "scale", dt)
    if _mod_rows(shift, B, D, "shift", dt) != bs:
        raise ValueError("scale and shift must share one batch stride")
    out = _out_like(out, y)
    _call(entry, _ptr(y), _ptr(scale), _ptr(shift), _ptr(out), B, S, D, bs, _stream(stream))
    return out


def residual_gate_add(residual, gate, update, out=None, stream=None):
    """R(residual + R(gate * update)) over [B, S, D]."""
    B, S, D = _bsd(residual, "residual")
    _dense(update, "update")
    if update.shape != residual.shape:
        raise ValueError("update must match residual")
    gs = _mod_rows(gate, B, D, "gate")
    out = _out_like(out, residual)
    _call("residual_gate_add", _ptr(residual), _ptr(gate), _ptr(update), gs, _ptr(out), B, S, D,
          _stream(stream))
    return out


def conv_bias_epilogue(x, bias, h=None, out=None, stream=None):
    """R(x + R(bias)) (and + h) on a channels-last activation."""
    _bf16(x, "x")
    pixels, C = _pixels_c(x)
    if bias.dtype not in (torch.float32, torch.bfloat16) or not bias.is_cuda or \
            bias.numel() != C or not bias.is_contiguous():
        raise ValueError("bias must be a contiguous fp32/bf16 CUDA tensor of C elements")
    if h is not None:
        _bf16(h, "h")
        if h.shape != x.shape or h.stride() != x.stride():
            raise ValueError("h must match x's shape and strides")
    if out is None:
        out = torch.empty_like(x)
    is32 = 1 if bias.dtype == torch.float32 else 0
    _call("conv_bias_epilogue", _ptr(x), _ptr(bias), is32, _ptr(h), _ptr(out), pixels, C,
          _stream(stream))
    return out


_DTYPES = {torch.bfloat16: 0, torch.float16: 1}

# Checks of the calls below.  They take most of a small call's time, so each reads an attribute once
# and leaves the wording of an error to the end.


def _half(t, name):
    if isinstance(t, torch.Tensor) and t.dtype in _DTYPES and t.is_cuda and t.is_contiguous():
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float16, got {t.dtype}")
    return _dense(t, name, t.dtype)


def _input(t, name, dtype, device, shape):
    """A required contiguous tensor."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and \
            t.device == device and t.is_contiguous():
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} shape {tuple(t.shape)} != {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _vector(t, name, dtype, device, D):
    """A nullable vector of D elements."""
    if t is None or (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == D and
                     t.device == device and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.numel() != D:
        raise ValueError(f"{name} must have {D} elements")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _rows(t, name, dtype, device, B, D):
    """Batch stride of a nullable modulation row (0 = shared by every batch)."""
    if t is None:
        return 0
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.device == device:
        shape = t.shape
        if len(shape) == 3 and shape[0] == B and shape[1] == 1 and shape[2] == D:
            stride = t.stride()
            if stride[2] == 1:
                return stride[0] if B > 1 else 0
    elif isinstance(t, torch.Tensor) and t.dtype is dtype:
        raise ValueError(f"{name} must be on {device}")
    return _mod_rows(t, B, D, name, dtype)


def _modulation(scale, shift, dtype, device, B, D):
    """Batch stride of the nullable scale and shift rows."""
    bs = _rows(scale, "scale", dtype, device, B, D)
    if shift is not None:
        if scale is None:
            return _rows(shift, "shift", dtype, device, B, D)
        if (not isinstance(shift, torch.Tensor) or shift.dtype is not dtype or
                shift.device != device or shift.shape != scale.shape or
                shift.stride() != scale.stride()) and \
                _rows(shift, "shift", dtype, device, B, D) != bs:
            raise ValueError("scale and shift must share one batch stride")
    return bs


def _stats(t, name, device, n):
    """Nullable fp32 statistics of n rows."""
    if t is not None and (t.dtype is not torch.float32 or t.numel() != n or t.device != device or
                          not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous float32 tensor of {n} elements on {device}")


def sandwich_rmsnorm_modulate(residual, update, post_weight=None, gate=None, weight=None,
                              scale=None, shift=None, eps: float = 1e-6, post_eps=None,
                              residual_scale: float = 1.0, update_scale: float = 1.0,
                              need_out=True, res_out=None, out=None, post_rstd_out=None,
                              rstd_out=None, stream=None):
    """The norm after a block with its gate and residual scale, the residual add, and the norm
    before the next block:

        res = R(residual_scale * residual + update_scale * gate * RMSNorm(update) * post_weight)
        out = R(RMSNorm(res) * weight * (1 + scale) + shift)

    -> (res, out); out is None without need_out.  bfloat16 or float16, one rounding per value.
    A missing post_weight, gate, weight or scale is a factor of 1, a missing shift 0; post_eps
    defaults to eps.  post_rstd_out / rstd_out: fp32 [B * S] for the backward pass."""
    _half(residual, "residual")
    dt, device, shape = residual.dtype, residual.device, residual.shape
    if stream is not None and (res_out is None or (need_out and out is None)):
        return _aside(stream, device, sandwich_rmsnorm_modulate, residual, update, post_weight, gate,
                      weight, scale, shift, eps, post_eps, residual_scale, update_scale, need_out,
                      res_out, out, post_rstd_out, rstd_out)
    B, S, D = shape if len(shape) == 3 else _bsd(residual, "residual", dt)
    _input(update, "update", dt, device, shape)
    _vector(post_weight, "post_weight", dt, device, D)
    gs = _rows(gate, "gate", dt, device, B, D)
    if not need_out and (out is not None or rstd_out is not None):
        raise ValueError("out and rstd_out need need_out")
    _vector(weight, "weight", dt, device, D)
    bs = _modulation(scale, shift, dt, device, B, D)
    if res_out is None:
        res_out = torch.empty_like(residual)
    else:
        _input(res_out, "res_out", dt, device, shape)
    if out is not None:
        _input(out, "out", dt, device, shape)
    elif need_out:
        out = torch.empty_like(residual)
    _stats(post_rstd_out, "post_rstd_out", device, B * S)
    _stats(rstd_out, "rstd_out", device, B * S)
    _call_on(device, stream, "sandwich_rmsnorm_modulate", _at(residual), _at(update), _at(post_weight),
             _at(gate), gs, _at(weight), _at(scale), _at(shift), bs, _at(res_out), _at(out), B, S, D,
             residual_scale, update_scale, eps if post_eps is None else post_eps, eps,
             _at(post_rstd_out), _at(rstd_out), _DTYPES[dt])
    return res_out, out


class SandwichGrads(NamedTuple):
    """Gradients of sandwich_rmsnorm_modulate by its inputs: residual and update of their type,
    the row vectors in fp32 ([D]; gate, scale and shift [B, D], or [1, D] where one row is shared
    by the batches); None for an input that took no part (a gradient of shift comes with that of
    scale, whether or not the call was given shift)."""

    residual: torch.Tensor
    update: torch.Tensor
    post_weight: torch.Tensor
    gate: torch.Tensor
    weight: torch.Tensor
    scale: torch.Tensor
    shift: torch.Tensor


def _row_grads(wanted, stride, B, D, device):
    if not wanted:
        return None
    return torch.empty(B if stride else 1, D, dtype=torch.float32, device=device)


def _vector_grad(wanted, D, device):
    return torch.empty(D, dtype=torch.float32, device=device) if wanted else None


def _need_stats(t, name, device, n):
    if t is None:
        raise ValueError(f"{name} (the forward's statistics) is required")
    _stats(t, name, device, n)


@functools.lru_cache(maxsize=256)
def _workspace_bytes(name, B, S, D):
    return int(getattr(library(), name + "_workspace_bytes")(B, S, D))


def _backward_workspace(name, workspace, wanted, B, S, D, device):
    if not wanted:
        return None, 0
    need = _workspace_bytes(name, B, S, D)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {device}")
    wbytes = workspace.numel() * workspace.element_size()
    if wbytes < need:
        raise ValueError(f"workspace holds fewer than the {need} bytes needed")
    return workspace, wbytes


def sandwich_rmsnorm_modulate_backward(update, res, post_weight, gate, weight, scale, grad_res,
                                       grad_out, post_rstd, rstd, residual_scale: float = 1.0,
                                       update_scale: float = 1.0, need_x=True, need_mod=True,
                                       workspace=None, stream=None, shift=None) -> SandwichGrads:
    """Gradients of sandwich_rmsnorm_modulate.  update, post_weight, gate, weight, scale and the
    two factors as in the forward, res and the statistics as it left them; grad_res, grad_out: the
    gradients of res and out (grad_res may be None; without grad_out, which drops the second norm,
    grad_res is needed and res, weight, scale, shift and rstd are not).  need_x: residual and
    update; need_mod: the row vectors, whose token sums (in an order that S and D fix) take a
    workspace, allocated here unless one is passed.  A gradient of shift comes with that of scale;
    where the forward had shift and no scale, it is given here too (its rows' shape and stride are
    read, its values are not)."""
    _half(update, "update")
    dt, device, shape = update.dtype, update.device, update.shape
    if stream is not None:
        return _aside(stream, device, functools.partial(sandwich_rmsnorm_modulate_backward,
                                                        shift=shift),
                      update, res, post_weight, gate, weight, scale, grad_res, grad_out, post_rstd,
                      rstd, residual_scale, update_scale, need_x, need_mod, workspace)
    B, S, D = shape if len(shape) == 3 else _bsd(update, "update", dt)
    if grad_res is not None:
        _input(grad_res, "grad_res", dt, device, shape)
    elif grad_out is None:
        raise ValueError("grad_res or grad_out is required")
    _vector(post_weight, "post_weight", dt, device, D)
    gs = _rows(gate, "gate", dt, device, B, D)
    bs = 0
    _need_stats(post_rstd, "post_rstd", device, B * S)
    if grad_out is not None:
        _input(grad_out, "grad_out", dt, device, shape)
        if res is None:
            raise ValueError("res is required with grad_out")
        _input(res, "res", dt, device, shape)
        _vector(weight, "weight", dt, device, D)
        bs = _modulation(scale, shift, dt, device, B, D)
        _need_stats(rstd, "rstd", device, B * S)
    else:
        res = weight = scale = shift = rstd = None
    g = SandwichGrads(
        torch.empty_like(update) if need_x else None,
        torch.empty_like(update) if need_x else None,
        _vector_grad(need_mod and post_weight is not None, D, device),
        _row_grads(need_mod and gate is not None, gs, B, D, device),
        _vector_grad(need_mod and weight is not None, D, device),
        _row_grads(need_mod and scale is not None, bs, B, D, device),
        _row_grads(need_mod and (scale is not None or shift is not None), bs, B, D, device))
    workspace, wbytes = _backward_workspace("sandwich_rmsnorm_modulate_backward", workspace,
                                            need_mod, B, S, D, device)
    _call_on(device, stream, "sandwich_rmsnorm_modulate_backward", _at(update), _at(res),
             _at(post_weight), _at(gate), gs, _at(weight), _at(scale), bs, _at(grad_res),
             _at(grad_out), _at(post_rstd), _at(rstd), B, S, D, residual_scale, update_scale,
             _at(g.residual), _at(g.update), _at(g.post_weight), _at(g.gate), _at(g.weight),
             _at(g.scale), _at(g.shift), _at(workspace), wbytes, _DTYPES[dt])
    return g


def rmsnorm_modulate_backward(x, weight, scale, grad_out, rstd, grad_res=None, need_x=True,
                              need_mod=True, workspace=None, stream=None):
    """Gradients of rmsnorm_modulate (bfloat16; x, weight, scale as in the forward, rstd its
    statistics) -> (grad_x, grad_weight, grad_scale, grad_shift).  grad_res: a gradient that
    reaches x on the residual stream, added to grad_x before its rounding.  grad_weight fp32 [D];
    grad_scale, grad_shift fp32 [B, D] ([1, D] where one row is shared); scale may be None (no
    modulation: no such gradients).  Workspace as in sandwich_rmsnorm_modulate_backward."""
    _dense(x, "x", torch.bfloat16)
    dt, device, shape = x.dtype, x.device, x.shape
    if stream is not None:
        return _aside(stream, device, rmsnorm_modulate_backward, x, weight, scale, grad_out, rstd,
                      grad_res, need_x, need_mod, workspace)
    B, S, D = shape if len(shape) == 3 else _bsd(x)
    _input(grad_out, "grad_out", dt, device, shape)
    if grad_res is not None:
        _input(grad_res, "grad_res", dt, device, shape)
    _vector(weight, "weight", dt, device, D)
    bs = _rows(scale, "scale", dt, device, B, D)
    _need_stats(rstd, "rstd", device, B * S)
    grad_x = torch.empty_like(x) if need_x else None
    grad_weight = _vector_grad(need_mod and weight is not None, D, x.device)
    grad_scale = _row_grads(need_mod and scale is not None, bs, B, D, x.device)
    grad_shift = _row_grads(need_mod and scale is not None, bs, B, D, x.device)
    workspace, wbytes = _backward_workspace("rmsnorm_modulate_backward", workspace, need_mod, B,
                                            S, D, x.device)
    _call_on(x.device, stream, "rmsnorm_modulate_backward", _at(x), _at(weight), _at(scale), bs,
             _at(grad_out), _at(grad_res), _at(rstd), B, S, D, _at(grad_x),
             _at(grad_weight), _at(grad_scale), _at(grad_shift), _at(workspace), wbytes)
    return grad_x, grad_weight, grad_scale, grad_shift


class Mxfp4(NamedTuple):
    """A microscaled 4-bit matrix: `packed` uint8 [..., K / 2] (two e2m1 codes a byte, the even
    element in the low half) and `scales` uint8, the tiled e8m0 scale bytes of its rows
    (mxfp4_scale_bytes(rows, K) of them; layout in include/rmsmod.h)."""

    packed: torch.Tensor
    scales: torch.Tensor


@functools.lru_cache(maxsize=256)
def mxfp4_scale_bytes(rows: int, K: int) -> int:
    """Bytes of the tiled scales of a [rows, K] 4-bit matrix (0 if the size is unsupported)."""
    return int(library().mxfp4_scale_bytes(rows, K))


def _codes(q, name, device=None):
    """-> (rows, K) of a checked Mxfp4."""
    if not isinstance(q, Mxfp4):
        raise TypeError(f"{name} must be an Mxfp4")
    packed, scales = q
    _dense(packed, f"{name}.packed", torch.uint8)
    _dense(scales, f"{name}.scales", torch.uint8)
    if packed.device != scales.device or (device is not None and packed.device != device):
        raise ValueError(f"{name} must be on {packed.device if device is None else device}")
    shape = packed.shape
    K = 2 * shape[-1] if shape else 0
    if K == 0 or K % 32:
        raise ValueError(f"{name}.packed must hold rows of a multiple of 32 values")
    rows = 2 * packed.numel() // K
    if scales.numel() != mxfp4_scale_bytes(rows, K):
        raise ValueError(f"{name}.scales must hold {mxfp4_scale_bytes(rows, K)} bytes")
    return rows, K


def mxfp4_quantize(x, out=None, stream=None) -> Mxfp4:
    """Rows of x [..., K] (bfloat16 or float16, K a multiple of 32) in blocks of 32 e2m1 codes
    under the least power-of-two scale that holds the block without saturation."""
    _half(x, "x")
    if stream is not None and out is None:
        return _aside(stream, x.device, mxfp4_quantize, x, out)
    K = x.shape[-1] if x.dim() else 0
    if K == 0 or K % 32:
        raise ValueError("x must hold rows of a multiple of 32 values")
    rows = x.numel() // K
    if out is None:
        out = Mxfp4(torch.empty(*x.shape[:-1], K // 2, dtype=torch.uint8, device=x.device),
                    torch.empty(mxfp4_scale_bytes(rows, K), dtype=torch.uint8, device=x.device))
    elif _codes(out, "out", x.device) != (rows, K):
        raise ValueError("out must match x")
    _call_on(x.device, stream, "mxfp4_quantize", _at(x), _at(out.packed), _at(out.scales), rows, K,
             _DTYPES[x.dtype])
    return out


def mxfp4_dequantize(q, dtype=torch.bfloat16, out=None, stream=None):
    """The values that q stands for, as bfloat16 or float16 [..., K]."""
    rows, K = _codes(q, "q")
    if stream is not None and out is None:
        return _aside(stream, q.packed.device, mxfp4_dequantize, q, dtype, out)
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
    if out is None:
        out = torch.empty(*q.packed.shape[:-1], K, dtype=dtype, device=q.packed.device)
    else:
        _dense(out, "out", dtype)
        if out.shape != (*q.packed.shape[:-1], K) or out.device != q.packed.device:
            raise ValueError("out must match q")
    _call_on(out.device, stream, "mxfp4_dequantize", _at(q.packed), _at(q.scales), _at(out), rows, K,
             _DTYPES[dtype])
    return out


def mxfp4_linear(x, w, bias=None, gate=None, residual=None, out=None, dtype=None, stream=None):
    """x w^T in 4 bits, its bias, and a block's gated residual add in the epilogue:
    R(residual + gate * (x w^T + bias)), one rounding.

    x [..., K]: bfloat16 or float16 (quantised here) or an Mxfp4 (then `dtype`, default
    bfloat16, is the result's type); w: an Mxfp4 [N, K], laid out once.  bias [N]; gate rows [N]
    or [B, 1, N] (for x [B, S, K]); residual [..., N], all of the result's type.  out may be
    residual."""
    if stream is not None and (out is None or not isinstance(x, Mxfp4)):
        at = x.packed if isinstance(x, Mxfp4) else x
        if not isinstance(at, torch.Tensor):
            raise TypeError("x must be a torch.Tensor or an Mxfp4")
        return _aside(stream, at.device, mxfp4_linear, x, w, bias, gate, residual, out, dtype)
    if isinstance(x, Mxfp4):
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in _DTYPES:
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        width = _codes(x, "x")[1]
        lead, device = x.packed.shape[:-1], x.packed.device
    else:
        _half(x, "x")
        if dtype is not None and dtype != x.dtype:
            raise TypeError(f"dtype must be x's, {x.dtype}")
        dtype, lead, device = x.dtype, x.shape[:-1], x.device
        width = x.shape[-1] if x.dim() else 0
    N, K = _codes(w, "w", device)
    if w.packed.dim() != 2 or N % 8:
        raise ValueError("w must be [N, K], N a multiple of 8")
    if len(lead) == 0 or width != K:
        raise ValueError(f"x must hold rows of K={K} values")
    B = lead[0] if len(lead) > 1 else 1
    M = 1
    for n in lead:
        M *= n
    S = M // B if B else 0
    _vector(bias, "bias", dtype, device, N)
    gs = _rows(gate, "gate", dtype, device, B, N)
    shape = (*lead, N)
    if residual is not None:
        _input(residual, "residual", dtype, device, shape)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    else:
        _input(out, "out", dtype, device, shape)
    code = _DTYPES[dtype]
    if isinstance(x, Mxfp4):
        packed, scales = _at(x.packed), _at(x.scales)
    else:
        codes = M * (K // 2)  # a multiple of 16
        q = torch.empty(codes + mxfp4_scale_bytes(M, K), dtype=torch.uint8, device=device)
        packed = _at(q)
        scales = packed + codes
        _call_on(device, stream, "mxfp4_quantize", _at(x), packed, scales, M, K, code)
    _call_on(device, stream, "mxfp4_matmul", packed, scales, _at(w.packed), _at(w.scales), _at(bias),
             _at(gate), gs, _at(residual), _at(out), B, S, N, K, code)
    return out


class Mxfp8(NamedTuple):
    """A microscaled 8-bit matrix: `codes` torch.float8_e4m3fn [..., K] and `scales` uint8, the tiled
    e8m0 scale bytes of its rows (mxfp8_scale_bytes(rows, K) of them; layout in include/rmsmod.h)."""

    codes: torch.Tensor
    scales: torch.Tensor


_E4M3 = torch.float8_e4m3fn
_DIRECT_ROWS = 32  # RMSMOD_MXFP8_DIRECT_ROWS
_ACTIVATIONS = {None: 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


@functools.lru_cache(maxsize=256)
def mxfp8_scale_bytes(rows: int, K: int) -> int:
    """Bytes of the tiled scales of a [rows, K] 8-bit matrix (0 if the size is unsupported)."""
    return int(library().mxfp8_scale_bytes(rows, K))


def _codes8(q, name, device=None):
    """-> (rows, K) of a checked Mxfp8."""
    if not isinstance(q, Mxfp8):
        raise TypeError(f"{name} must be an Mxfp8")
    codes, scales = q
    if not (isinstance(codes, torch.Tensor) and isinstance(scales, torch.Tensor) and
            codes.dtype is _E4M3 and scales.dtype is torch.uint8 and codes.is_cuda and
            codes.is_contiguous() and scales.is_contiguous()):
        _dense(codes, f"{name}.codes", _E4M3)
        _dense(scales, f"{name}.scales", torch.uint8)
    at = codes.device
    if at != scales.device or (device is not None and at != device):
        raise ValueError(f"{name} must be on {at if device is None else device}")
    shape = codes.shape
    K = shape[-1] if shape else 0
    if K == 0 or K % 32:
        raise ValueError(f"{name}.codes must hold rows of a multiple of 32 values")
    rows = codes.numel() // K
    need = mxfp8_scale_bytes(rows, K)
    if scales.numel() != need:
        raise ValueError(f"{name}.scales must hold {need} bytes")
    return rows, K


def _new8(shape, rows, device):
    """An Mxfp8 to be written."""
    return Mxfp8(torch.empty(shape, dtype=_E4M3, device=device),
                 torch.empty(mxfp8_scale_bytes(rows, shape[-1]), dtype=torch.uint8, device=device))


def _out8(q, name, shape, device):
    """A checked Mxfp8 of that shape to write to."""
    _codes8(q, name, device)
    if q.codes.shape != shape:
        raise ValueError(f"{name}.codes shape {tuple(q.codes.shape)} != {tuple(shape)}")
    return q


def _written_over(x, *outs):
    """Whether one of the given outputs (tensors, Mxfp8 or None) has bytes of the contiguous x."""
    begin = x.data_ptr()
    end = begin + x.numel() * x.element_size()
    for t in outs:
        if isinstance(t, Mxfp8):
            if _written_over(x, *t):
                return True
        elif t is not None:
            at = t.data_ptr()
            if at < end and begin < at + t.numel() * t.element_size():
                return True
    return False


def _activation(name):
    code = _ACTIVATIONS.get(name) if name is None or isinstance(name, str) else None
    if code is None:
        raise ValueError(f"activation must be None, 'silu', 'gelu' or 'gelu_tanh', got {name!r}")
    return code


def mxfp8_quantize(x, out=None, stream=None) -> Mxfp8:
    """Rows of x [..., K] (bfloat16 or float16, K a multiple of 32) in blocks of 32 e4m3 codes
    under the least power-of-two scale that holds the block without saturation."""
    _half(x, "x")
    if stream is not None and out is None:
        return _aside(stream, x.device, mxfp8_quantize, x, out)
    K = x.shape[-1] if x.dim() else 0
    if K == 0 or K % 32:
        raise ValueError("x must hold rows of a multiple of 32 values")
    rows = x.numel() // K
    if out is None:
        out = _new8(x.shape, rows, x.device)
    else:
        _out8(out, "out", x.shape, x.device)
    _call_on(x.device, stream, "mxfp8_quantize", _at(x), _at(out.codes), _at(out.scales), rows, K,
             _DTYPES[x.dtype])
    return out


def mxfp8_dequantize(q, dtype=torch.bfloat16, out=None, stream=None):
    """The values that q stands for, as bfloat16 or float16 [..., K]."""
    rows, K = _codes8(q, "q")
    if stream is not None and out is None:
        return _aside(stream, q.codes.device, mxfp8_dequantize, q, dtype, out)
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
    if out is None:
        out = torch.empty(q.codes.shape, dtype=dtype, device=q.codes.device)
    else:
        _input(out, "out", dtype, q.codes.device, q.codes.shape)
    _call_on(out.device, stream, "mxfp8_dequantize", _at(q.codes), _at(q.scales), _at(out), rows, K,
             _DTYPES[dtype])
    return out


def mxfp8_transpose(q, out=None, stream=None) -> Mxfp8:
    """The matrix q [..., K] of R rows as [K, R up to a multiple of 32], in blocks along its rows
    (zeros behind the last one): what a weight's gradient takes of an activation and of its
    gradient, and an input's gradient of a weight.  A value keeps its bits but where it is under 2^-6
    of its new block's scale."""
    rows, K = _codes8(q, "q")
    device = q.codes.device
    if stream is not None and out is None:
        return _aside(stream, device, mxfp8_transpose, q, out)
    shape = (K, -(-rows // 32) * 32)
    if out is None:
        if not rows:
            raise ValueError("q must have rows")
        out = _new8(shape, K, device)
    else:
        _out8(out, "out", shape, device)
    _call_on(device, stream, "mxfp8_transpose", _at(q.codes), _at(q.scales), _at(out.codes),
             _at(out.scales), rows, K)
    return out


def mxfp8_linear(x, w, bias=None, activation=None, gate=None, residual=None, out=None, dtype=None,
                 quantize=False, keep=False, stream=None):
    """A projection in 8 bits with its epilogue:

        z = x w^T + bias,  y = residual + gate * act(z)

    -> y, rounded once, or with `quantize` as an Mxfp8 in blocks along N; with `keep` (y, z), z an
    Mxfp8 for mxfp8_activation_backward.

    x [..., K]: bfloat16 or float16 (quantised here) or an Mxfp8 (then `dtype`, default bfloat16, is
    the type of the result, bias, gate and residual; torch.float32 too, for a weight's gradient); w:
    an Mxfp8 [N, K].  activation: None, "silu", "gelu" or "gelu_tanh", good to (16 + 4 |ln p|) 2^-24
    of itself with p = act(z) / z (2^-19 for z >= 0) whatever the dtype.  bias [N]; gate rows [N] or
    [B, 1, N] (for x [B, S, K]); residual [..., N].  N a multiple of 8, of 32 with `quantize` or
    `keep`.  out (of y) may be residual; keep may be the Mxfp8 to write z to; either may lie in a 16-bit
    x, which is quantised before."""
    if stream is not None and (out is None or keep is True or not isinstance(x, Mxfp8)):
        at = x.codes if isinstance(x, Mxfp8) else x
        if not isinstance(at, torch.Tensor):
            raise TypeError("x must be a torch.Tensor or an Mxfp8")
        return _aside(stream, at.device, mxfp8_linear, x, w, bias, activation, gate, residual, out,
                      dtype, quantize, keep)
    if isinstance(x, Mxfp8):
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in _DTYPES and dtype != torch.float32:
            raise TypeError("dtype must be torch.bfloat16, torch.float16 or torch.float32, "
                            f"got {dtype}")
        width = _codes8(x, "x")[1]
        lead, device = x.codes.shape[:-1], x.codes.device
    else:
        _half(x, "x")
        if dtype is not None and dtype != x.dtype:
            raise TypeError(f"dtype must be x's, {x.dtype}")
        dtype, lead, device = x.dtype, x.shape[:-1], x.device
        width = x.shape[-1] if x.dim() else 0
    act = _activation(activation)
    N, K = _codes8(w, "w", device)
    eight = quantize or bool(keep)
    if w.codes.dim() != 2 or N % (32 if eight else 8):
        raise ValueError(f"w must be [N, K], N a multiple of {32 if eight else 8}")
    if len(lead) == 0 or width != K:
        raise ValueError(f"x must hold rows of K={K} values")
    B = lead[0] if len(lead) > 1 else 1
    M = 1
    for n in lead:
        M *= n
    S = M // B if B else 0
    _vector(bias, "bias", dtype, device, N)
    gs = _rows(gate, "gate", dtype, device, B, N)
    shape = (*lead, N)
    if residual is not None:
        _input(residual, "residual", dtype, device, shape)
    fresh = out is None and not isinstance(keep, Mxfp8)
    if quantize:
        out = _new8(shape, M, device) if out is None else _out8(out, "out", shape, device)
        y, y_scales = _at(out.codes), _at(out.scales)
    else:
        if out is None:
            out = torch.empty(shape, dtype=dtype, device=device)
        else:
            _input(out, "out", dtype, device, shape)
        y, y_scales = _at(out), None
    kept = None
    if keep is True:
        kept = _new8(shape, M, device)
    elif keep:
        kept = _out8(keep, "keep", shape, device)
    code = 2 if dtype == torch.float32 else _DTYPES[dtype]
    if isinstance(x, Mxfp8):
        codes, scales = _at(x.codes), _at(x.scales)
    elif M <= _DIRECT_ROWS and (fresh or not _written_over(x, out, kept)):
        codes, scales = _at(x), None  # quantised by the product itself, which does not write to it
    else:
        n = M * K  # a multiple of 32
        q = torch.empty(n + mxfp8_scale_bytes(M, K), dtype=torch.uint8, device=device)
        codes = _at(q)
        scales = codes + n
        _call_on(device, stream, "mxfp8_quantize", _at(x), codes, scales, M, K, code)
    _call_on(device, stream, "mxfp8_matmul", codes, scales, _at(w.codes), _at(w.scales), _at(bias),
             act, _at(gate), gs, _at(residual), y, y_scales,
             None if kept is None else _at(kept.codes),
             None if kept is None else _at(kept.scales), B, S, N, K, code)
    return out if kept is None else (out, kept)


def mxfp8_activation_backward(z, grad_out, activation=None, gate=None, need_sums=True, out=None,
                              workspace=None, stream=None):
    """Gradients of y = residual + gate * act(z), z = x w^T + bias, from the checkpoint z [..., N] of
    mxfp8_linear and grad_out, the gradient of y (bfloat16 or float16): -> (grad_z, grad_bias,
    grad_gate), grad_z = Q(grad_out * gate * act'(z)) an Mxfp8, grad_bias fp32 [N] (the sum of
    grad_z's values before Q), grad_gate fp32 [B, N] ([1, N] where one row is shared), None without
    gate.  The sums (in an order that the sizes fix) take a workspace, allocated here unless one is
    passed; both are None without need_sums.

    Then the gradients of x and w are products of 8-bit rows again:
    mxfp8_linear(grad_z, mxfp8_transpose(w)) and
    mxfp8_linear(mxfp8_transpose(grad_z), mxfp8_transpose(x), dtype=torch.float32)."""
    if stream is not None:
        if not isinstance(z, Mxfp8):
            raise TypeError("z must be an Mxfp8")
        return _aside(stream, z.codes.device, mxfp8_activation_backward, z, grad_out, activation,
                      gate, need_sums, out, workspace)
    rows, N = _codes8(z, "z")
    device, shape = z.codes.device, z.codes.shape
    _half(grad_out, "grad_out")
    dt = grad_out.dtype
    _input(grad_out, "grad_out", dt, device, shape)
    act = _activation(activation)
    B = shape[0] if len(shape) > 2 else 1
    S = rows // B if B else 0
    gs = _rows(gate, "gate", dt, device, B, N)
    out = _new8(shape, rows, device) if out is None else _out8(out, "out", shape, device)
    grad_bias = _vector_grad(need_sums, N, device)
    grad_gate = _row_grads(need_sums and gate is not None, gs, B, N, device)
    workspace, wbytes = _backward_workspace("mxfp8_activation_backward", workspace, need_sums,
                                            *((B, S) if gs else (1, rows)), N, device)
    _call_on(device, stream, "mxfp8_activation_backward", _at(z.codes), _at(z.scales),
             _at(grad_out), act, _at(gate), gs, _at(out.codes), _at(out.scales), _at(grad_bias),
             _at(grad_gate), B, S, N, _at(workspace), wbytes, _DTYPES[dt])
    return out, grad_bias, grad_gate


def add_rmsnorm_mxfp8(x, update=None, weight=None, scale=None, shift=None, eps: float = 1e-6,
                      keep=False, res_out=None, out=None, rstd_out=None, stream=None):
    """The residual add and the norm before a projection in 8 bits:

        res = R(x + update),  out = Q(RMSNorm(res) * weight * (1 + scale) + shift)

    -> (res, out, kept): out an Mxfp8 for mxfp8_linear, rounded from fp32 once; kept = Q(res) with
    `keep` (True, or the Mxfp8 to write to), the checkpoint that rmsnorm_mxfp8_backward takes, else
    None.  bfloat16 or float16, rows of a multiple of 32 values.  Without update res is x itself.  A
    missing weight or scale is a factor of 1, a missing shift 0.  res_out may be x or update.
    rstd_out: fp32 [B * S] for the backward pass."""
    _half(x, "x")
    dt, device, shape = x.dtype, x.device, x.shape
    if stream is not None and (out is None or keep is True or
                               (update is not None and res_out is None)):
        made = _aside(stream, device, _add_rmsnorm_mxfp8_made, x, update, weight, scale, shift, eps,
                      keep, res_out, out, rstd_out)
        return (x, *made[1:]) if update is None else made
    B, S, D = shape if len(shape) == 3 else _bsd(x, "x", dt)
    if D % 32:
        raise ValueError("x must hold rows of a multiple of 32 values")
    if update is not None:
        _input(update, "update", dt, device, shape)
    elif res_out is not None:
        raise ValueError("res_out needs update")
    _vector(weight, "weight", dt, device, D)
    bs = _modulation(scale, shift, dt, device, B, D)
    res = x
    if update is not None:
        if res_out is None:
            res_out = torch.empty_like(x)
        else:
            _input(res_out, "res_out", dt, device, shape)
        res = res_out
    rows = B * S
    out = _new8(shape, rows, device) if out is None else _out8(out, "out", shape, device)
    kept = None
    if keep is True:
        kept = _new8(shape, rows, device)
    elif keep:
        kept = _out8(keep, "keep", shape, device)
    _stats(rstd_out, "rstd_out", device, rows)
    _call_on(device, stream, "add_rmsnorm_mxfp8", _at(x), _at(update), _at(weight), _at(scale),
             _at(shift), bs, _at(res_out), _at(out.codes), _at(out.scales),
             None if kept is None else _at(kept.codes),
             None if kept is None else _at(kept.scales), B, S, D, eps, _at(rstd_out), _DTYPES[dt])
    return res, out, kept


def _add_rmsnorm_mxfp8_made(x, update, *args):
    """add_rmsnorm_mxfp8's results without x among them: what another stream has made."""
    res, out, kept = add_rmsnorm_mxfp8(x, update, *args)
    return None if update is None else res, out, kept


def rmsnorm_mxfp8_backward(kept, weight, scale, grad_out, rstd, grad_res=None, need_x=True,
                           need_mod=True, workspace=None, stream=None, shift=None):
    """Gradients of add_rmsnorm_mxfp8 (weight, scale as in the forward; kept and rstd as it left
    them) -> (grad_x, grad_weight, grad_scale, grad_shift), grad_x by x and by update alike.
    grad_out: the gradient of out; grad_res: one that reaches res on the residual stream, added to
    grad_x before its rounding.  grad_weight fp32 [D]; grad_scale, grad_shift fp32 [B, D] ([1, D]
    where one row is shared), None without scale; where the forward had shift and no scale, it is
    given here too (its rows' shape and stride are read, its values are not).  Workspace as in
    sandwich_rmsnorm_modulate_backward."""
    if stream is not None:
        if not isinstance(kept, Mxfp8):
            raise TypeError("kept must be an Mxfp8")
        return _aside(stream, kept.codes.device,
                      functools.partial(rmsnorm_mxfp8_backward, shift=shift), kept, weight, scale,
                      grad_out, rstd, grad_res, need_x, need_mod, workspace)
    rows, D = _codes8(kept, "kept")
    device, shape = kept.codes.device, kept.codes.shape
    _half(grad_out, "grad_out")
    dt = grad_out.dtype
    _input(grad_out, "grad_out", dt, device, shape)
    if len(shape) != 3 and len(shape) != 2:
        raise ValueError("kept must be [B, S, D] or [S, D]")
    B = shape[0] if len(shape) == 3 else 1
    S = shape[-2]
    if grad_res is not None:
        _input(grad_res, "grad_res", dt, device, shape)
    _vector(weight, "weight", dt, device, D)
    bs = _modulation(scale, shift, dt, device, B, D)
    _need_stats(rstd, "rstd", device, rows)
    grad_x = torch.empty_like(grad_out) if need_x else None
    grad_weight = _vector_grad(need_mod and weight is not None, D, device)
    grad_scale = _row_grads(need_mod and scale is not None, bs, B, D, device)
    grad_shift = _row_grads(need_mod and (scale is not None or shift is not None), bs, B, D, device)
    workspace, wbytes = _backward_workspace("rmsnorm_mxfp8_backward", workspace, need_mod,
                                            *((B, S) if bs else (1, rows)), D, device)
    _call_on(device, stream, "rmsnorm_mxfp8_backward", _at(kept.codes), _at(kept.scales),
             _at(weight), _at(scale), bs, _at(grad_out), _at(grad_res), _at(rstd), B, S, D,
             _at(grad_x), _at(grad_weight), _at(grad_scale), _at(grad_shift), _at(workspace), wbytes,
             _DTYPES[dt])
    return grad_x, grad_weight, grad_scale, grad_shift


def device_status(clear: bool = False) -> int:
    """Error bits recorded by kernels on the current device (0 = none).
    Synchronous.  Bit 0: an asynchronous copy timed out (output invalid)."""
    bits = ctypes.c_uint(0)
    _call("rmsmod_device_status", ctypes.byref(bits), 1 if clear else 0)
    return int(bits.value)


def selftest_wait_timeout(limit_ns: int = 1_000_000, stream=None) -> None:
    """Launch the library's bounded-wait self-test: one warp waits `limit_ns`
    on a barrier nothing completes, then sets bit 0 of the device error word
    (read it with device_status after synchronising)."""
    _call("rmsmod_selftest_wait_timeout", int(limit_ns), _stream(stream))


def supported(op: int, d_or_c: int, *tensors) -> bool:
    """The library's predicate: never raises, never touches the GPU."""
    ptrs = (ctypes.c_void_p * max(1, len(tensors)))(
        *[t.data_ptr() if t is not None else None for t in tensors])
    return bool(library().rmsmod_supported(int(op), int(d_or_c), ptrs, len(tensors)))
