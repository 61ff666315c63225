"""Python face of the dense feed-forward sublayer (plain residual stream): argument checks and
marshalling over the C entry points of include/moe_ffn.h.

Every function enqueues on ``stream`` (default: the tensors' device's current stream) and returns
device tensors without waiting.  Outputs and workspaces that a call allocates belong to that stream.
Gradients come from explicit ``*_backward`` calls; nothing is recorded for autograd.  Rows may be
strided (``stride(-1) == 1``); weights and gates are contiguous.  Refused arguments raise
``ValueError`` (types, shapes) or ``MoeFFNError`` with the library's code.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import (ACTIVATIONS, GATE_NONE, GATE_TOKEN, GATE_VECTOR, MoeFfnBlockNormArgs, MoeFfnBlockNormGrads,
                   MoeFfnFp8MatmulArgs, MoeFfnFp8QuantiseArgs, MoeFfnGatedArgs)
from .api import MoeFFNError

_TYPES = {torch.float32: _lib.TYPE_F32, torch.bfloat16: _lib.TYPE_BF16, torch.float16: _lib.TYPE_F16}
_FP8 = {torch.float8_e4m3fn: _lib.TYPE_E4M3, torch.float8_e5m2: _lib.TYPE_E5M2}


# the current stream's handle of a device, by its index: torch.cuda.current_stream() makes a Stream
# object for it, which takes longer than the rest of a small call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _raise(rc: int):
    raise MoeFFNError(rc, _lib.load().moe_ffn_last_error(None).decode())


def _on(t: torch.Tensor, name: str, stream: Optional[torch.cuda.Stream]):
    """The context to run a call on tensor t in, or None where the current device and stream will do."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if stream is not None:
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, {name} on {t.device}")
        return torch.cuda.stream(stream)
    if index != torch.cuda.current_device():
        return torch.cuda.device(index)
    return None


# The checks below run on every call; they read each property of a tensor once.

def _matrix(name: str, t: torch.Tensor, index: int, shape, dtype) -> int:
    """Checks a matrix of `shape` on device `index`; returns the distance between its rows."""
    if t.shape != shape:
        raise ValueError(f"{name} must be of shape {list(shape)}, got {list(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on device {index}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return ld if shape[0] > 1 else shape[1]


def _whole(name: str, t: torch.Tensor, index: int, shape, dtype) -> int:
    """Checks a contiguous tensor of `shape`; returns its address."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on device {index}")
    return t.data_ptr()


def _shape2(name: str, t: torch.Tensor):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be [rows, columns], got {list(shape)}")
    return shape


def _norm_args(index, state, f, norm_f, gate, residual_scale, norm_next, eps, bt) -> MoeFfnBlockNormArgs:
    shape, ts = _shape2("state", state), state.dtype
    rows, hidden = shape
    if ts not in _TYPES or bt not in _TYPES or (ts is not torch.float32 and ts is not bt):
        raise ValueError("state must be float32 or of the block's type (float32, bfloat16, float16)")
    ld_state = _matrix("state", state, index, shape, ts)
    f_ptr = norm_f_ptr = norm_next_ptr = gate_ptr = None
    ld_f = gate_type = gate_kind = rows_per_gate = 0
    if f is not None:
        ld_f, f_ptr = _matrix("f", f, index, shape, bt), f.data_ptr()
    elif gate is not None or norm_f is not None:
        raise ValueError("gate and norm_f need f")
    if norm_f is not None:
        norm_f_ptr = _whole("norm_f", norm_f, index, (hidden,), torch.float32)
    if norm_next is not None:
        norm_next_ptr = _whole("norm_next", norm_next, index, (hidden,), torch.float32)
    if gate is not None:
        gs, gt = gate.shape, gate.dtype
        if gate.get_device() != index or (gt is not torch.float32 and gt is not bt) or not gate.is_contiguous():
            raise ValueError("gate must be contiguous, on the state's device, float32 or of the block's type")
        if gs == (hidden,):
            gate_kind, rows_per_gate = GATE_VECTOR, max(rows, 1)
        elif len(gs) == 2 and gs[1] == hidden and gs[0] > 0 and rows > 0 and rows % gs[0] == 0:
            gate_kind, rows_per_gate = GATE_VECTOR, rows // gs[0]
        elif gs == (rows, 1):
            gate_kind = GATE_TOKEN
        else:
            raise ValueError(f"gate must be [{hidden}], [G, {hidden}] with G dividing {rows}, or [{rows}, 1]; "
                             f"got {list(gs)}")
        gate_type, gate_ptr = _TYPES[gt], gate.data_ptr()
    return MoeFfnBlockNormArgs(rows, hidden, _TYPES[ts], _TYPES[bt], gate_type, gate_kind, rows_per_gate,
                               residual_scale, eps, state.data_ptr(), ld_state, f_ptr, ld_f, gate_ptr, norm_f_ptr,
                               norm_next_ptr)


def block_norm(state: torch.Tensor, f: Optional[torch.Tensor] = None, *, norm_f: Optional[torch.Tensor] = None,
               gate: Optional[torch.Tensor] = None, residual_scale: float = 1.0,
               norm_next: Optional[torch.Tensor] = None, eps: float = 1e-6, block_dtype: Optional[torch.dtype] = None,
               out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """The norms before and after a block, with the block's gate and residual scale, in one pass.

        n   = f * rsqrt(mean(f^2) + eps) * norm_f        (n = f without norm_f)
        out = state + residual_scale * gate * n
        y   = out * rsqrt(mean(out^2) + eps) * norm_next

    ``state`` [rows, hidden] float32 or of the block's type; ``f`` [rows, hidden], the block's output,
    float32, bfloat16 or float16; ``norm_f``, ``norm_next`` float32 [hidden]; ``gate`` [hidden],
    [G, hidden] (each row for rows / G consecutive rows) or [rows, 1].  Without ``f`` only y, the norm of
    ``state``, is made, in ``block_dtype`` (default: the state's type).  ``out`` may be ``state``.
    Returns (out, y); y is None without ``norm_next``, out is ``state`` itself without ``f``.
    """
    ctx = _on(state, "state", stream)
    if ctx is not None:
        with ctx:
            return block_norm(state, f, norm_f=norm_f, gate=gate, residual_scale=residual_scale, norm_next=norm_next,
                              eps=eps, block_dtype=block_dtype, out=out, y=y)
    bt = f.dtype if f is not None else (block_dtype or state.dtype)
    if block_dtype is not None and block_dtype != bt:
        raise ValueError("block_dtype must be f's type")
    index = state.get_device()
    a = _norm_args(index, state, f, norm_f, gate, residual_scale, norm_next, eps, bt)
    shape = state.shape
    if f is not None:
        if out is None:
            out, a.ld_out = torch.empty(shape, dtype=state.dtype, device=state.device), shape[1]
        else:
            a.ld_out = _matrix("out", out, index, shape, state.dtype)
        a.out = out.data_ptr()
    elif out is not None:
        raise ValueError("out is written only with f")
    if norm_next is not None:
        if y is None:
            y, a.ld_y = torch.empty(shape, dtype=bt, device=state.device), shape[1]
        else:
            a.ld_y = _matrix("y", y, index, shape, bt)
        a.y = y.data_ptr()
    elif y is not None:
        raise ValueError("y is written only with norm_next")
    rc = _lib.load().moe_ffn_block_norm(ctypes.byref(a), _raw_stream(index))
    if rc != 0:
        _raise(rc)
    return (out if f is not None else state), y


def block_norm_backward(out: torch.Tensor, f: Optional[torch.Tensor] = None, *,
                        norm_f: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                        residual_scale: float = 1.0, norm_next: Optional[torch.Tensor] = None, eps: float = 1e-6,
                        d_out: Optional[torch.Tensor] = None, d_y: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of :func:`block_norm`: ``out`` is what the forward call returned first (the stream after
    the block; without ``f`` the state), the other arguments are the forward call's.

    ``d_out`` (the stream's type) is the gradient that comes back along the stream, None for zero;
    ``d_y`` goes with ``norm_next``.  Returns a dict of the gradients of what was given: d_state, d_f,
    d_gate, d_norm_f and d_norm_next.
    """
    ctx = _on(out, "out", stream)
    if ctx is not None:
        with ctx:
            return block_norm_backward(out, f, norm_f=norm_f, gate=gate, residual_scale=residual_scale,
                                       norm_next=norm_next, eps=eps, d_out=d_out, d_y=d_y)
    if f is None and norm_next is None:
        raise ValueError("neither f nor norm_next is given")
    if (norm_next is None) != (d_y is None):
        raise ValueError("d_y goes with norm_next")
    index, dev, shape = out.get_device(), out.device, out.shape
    bt = f.dtype if f is not None else d_y.dtype
    a = _norm_args(index, out, f, norm_f, gate, residual_scale, norm_next, eps, bt)
    g, d = MoeFfnBlockNormGrads(), {}
    if d_out is not None:
        g.ld_d_out, g.d_out = _matrix("d_out", d_out, index, shape, out.dtype), d_out.data_ptr()
    if d_y is not None:
        g.ld_d_y, g.d_y = _matrix("d_y", d_y, index, shape, bt), d_y.data_ptr()

    def new(name, like_shape, dtype):
        d[name] = torch.empty(like_shape, dtype=dtype, device=dev)
        return d[name].data_ptr()

    g.d_state, g.ld_d_state = new("d_state", shape, out.dtype), shape[1]
    if f is not None:
        g.d_f, g.ld_d_f = new("d_f", shape, bt), shape[1]
    if gate is not None:
        g.d_gate = new("d_gate", gate.shape, gate.dtype)
    if norm_f is not None:
        g.d_norm_f = new("d_norm_f", (shape[1],), torch.float32)
    if norm_next is not None:
        g.d_norm_next = new("d_norm_next", (shape[1],), torch.float32)
    lib = _lib.load()
    need = lib.moe_ffn_block_norm_workspace(ctypes.byref(a), ctypes.byref(g))
    if need < 0:
        _raise(need)
    ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    if need:
        g.workspace, g.workspace_bytes = ws.data_ptr(), need
    rc = lib.moe_ffn_block_norm_backward(ctypes.byref(a), ctypes.byref(g), _raw_stream(index))
    if rc != 0:
        _raise(rc)
    return d


def _gated_args(index, x, w_gate, w_up, w_down, activation) -> MoeFfnGatedArgs:
    shape, dt = _shape2("x", x), x.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError("x must be bfloat16 or float16")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    rows, hidden = shape
    inter = _shape2("w_gate", w_gate)[0]
    return MoeFfnGatedArgs(rows, hidden, inter, _TYPES[dt], ACTIVATIONS[activation], x.data_ptr(),
                           _matrix("x", x, index, shape, dt), _whole("w_gate", w_gate, index, (inter, hidden), dt),
                           _whole("w_up", w_up, index, (inter, hidden), dt),
                           _whole("w_down", w_down, index, (hidden, inter), dt))


def _workspace(a: MoeFfnGatedArgs, need: int, device) -> torch.Tensor:
    if need < 0:
        _raise(need)
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    a.workspace, a.workspace_bytes = ws.data_ptr(), need
    return ws


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
              activation: str = "silu", save: bool = False, out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None):
    """The gated feed-forward block: y = (act(x w_gate^T) * (x w_up^T)) w_down^T.

    ``x`` [rows, hidden] bfloat16 or float16; ``w_gate``, ``w_up`` [inter, hidden] and ``w_down``
    [hidden, inter] of its type; hidden and inter multiples of 8.  ``activation``: "silu" or "gelu"
    (tanh form).  Returns y [rows, hidden]; with ``save`` also the pair (g, u) of projections
    [rows, inter] that :func:`gated_ffn_backward` takes.
    """
    ctx = _on(x, "x", stream)
    if ctx is not None:
        with ctx:
            return gated_ffn(x, w_gate, w_up, w_down, activation, save, out)
    index = x.get_device()
    a = _gated_args(index, x, w_gate, w_up, w_down, activation)
    if out is None:
        out, a.ld_y = torch.empty(x.shape, dtype=x.dtype, device=x.device), a.hidden
    else:
        a.ld_y = _matrix("out", out, index, x.shape, x.dtype)
    a.y = out.data_ptr()
    saved = None
    if save:
        saved = tuple(torch.empty((a.rows, a.inter), dtype=x.dtype, device=x.device) for _ in range(2))
        a.gate, a.up = saved[0].data_ptr(), saved[1].data_ptr()
    lib = _lib.load()
    ws = _workspace(a, lib.moe_ffn_gated_workspace(ctypes.byref(a), 0), x.device)  # noqa: F841
    rc = lib.moe_ffn_gated_forward(ctypes.byref(a), _raw_stream(index))
    if rc != 0:
        _raise(rc)
    return (out, saved) if save else out


def gated_ffn_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, saved,
                       d_y: torch.Tensor, activation: str = "silu", need_x: bool = True, need_weights: bool = True,
                       stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of :func:`gated_ffn` from what it saved: a dict of d_x, d_w_gate, d_w_up and d_w_down
    (of the inputs' type), without d_x or the weights' where they are not needed."""
    ctx = _on(x, "x", stream)
    if ctx is not None:
        with ctx:
            return gated_ffn_backward(x, w_gate, w_up, w_down, saved, d_y, activation, need_x, need_weights)
    index = x.get_device()
    a = _gated_args(index, x, w_gate, w_up, w_down, activation)
    a.gate, a.up = (_whole("saved", t, index, (a.rows, a.inter), x.dtype) for t in saved)
    a.ld_d_y, a.d_y = _matrix("d_y", d_y, index, x.shape, x.dtype), d_y.data_ptr()
    d = {}
    if need_x:
        d["d_x"] = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        a.d_x, a.ld_d_x = d["d_x"].data_ptr(), a.hidden
    if need_weights:
        for name, w in (("d_w_gate", w_gate), ("d_w_up", w_up), ("d_w_down", w_down)):
            d[name] = torch.empty_like(w)
            setattr(a, name, d[name].data_ptr())
    lib = _lib.load()
    ws = _workspace(a, lib.moe_ffn_gated_workspace(ctypes.byref(a), 1), x.device)  # noqa: F841
    rc = lib.moe_ffn_gated_backward(ctypes.byref(a), _raw_stream(index))
    if rc != 0:
        _raise(rc)
    return d


def fp8_quantise(x: torch.Tensor, block_rows: int = 1, pow2_scales: bool = False,
                 dtype: torch.dtype = torch.float8_e4m3fn, stream: Optional[torch.cuda.Stream] = None):
    """Makes an operand of :func:`fp8_matmul`: (codes [rows, k] of ``dtype``, float32 scales
    [ceil(rows / block_rows), ceil(k / 128)]).

    ``x`` [rows, k] float32, bfloat16 or float16.  ``block_rows`` 1 (activations) or 128 (weights).  A
    block's scale is its largest magnitude over the largest code, 1 for zeros, at least 2^-126, with
    ``pow2_scales`` rounded up to a power of two; a code is x * (1 / scale) rounded to nearest even.
    """
    ctx = _on(x, "x", stream)
    if ctx is not None:
        with ctx:
            return fp8_quantise(x, block_rows, pow2_scales, dtype)
    index = x.get_device()
    if x.dtype not in _TYPES or dtype not in _FP8:
        raise ValueError("x must be float32, bfloat16 or float16, dtype float8_e4m3fn or float8_e5m2")
    if block_rows not in (1, 128):
        raise ValueError("block_rows must be 1 or 128")
    rows, k = shape = _shape2("x", x)
    ld = _matrix("x", x, index, shape, x.dtype)
    codes = torch.empty((rows, k), dtype=dtype, device=x.device)
    scales = torch.empty((-(-rows // block_rows), -(-k // 128)), dtype=torch.float32, device=x.device)
    a = MoeFfnFp8QuantiseArgs(rows, k, _TYPES[x.dtype], _FP8[dtype], block_rows, bool(pow2_scales), x.data_ptr(), ld,
                              codes.data_ptr(), k, scales.data_ptr())
    rc = _lib.load().moe_ffn_fp8_quantise(ctypes.byref(a), _raw_stream(index))
    if rc != 0:
        _raise(rc)
    return codes, scales


def fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """a b^T of FP8 operands with float32 scales for blocks of 128: ``a`` [rows, k] with ``a_scale``
    [rows, ceil(k / 128)], ``b`` [n, k] with ``b_scale`` [ceil(n / 128), ceil(k / 128)] (see
    :func:`fp8_quantise`; each float8_e4m3fn or float8_e5m2), k a multiple of 16.  Sums are float32; the
    result is ``out_dtype``: float32, bfloat16 or float16.
    """
    ctx = _on(a, "a", stream)
    if ctx is not None:
        with ctx:
            return fp8_matmul(a, a_scale, b, b_scale, out_dtype, out)
    index, ta, tb = a.get_device(), a.dtype, b.dtype
    if ta not in _FP8 or tb not in _FP8 or out_dtype not in _TYPES:
        raise ValueError("a and b must be float8_e4m3fn or float8_e5m2, out_dtype float32, bfloat16 or float16")
    rows, k = shape = _shape2("a", a)
    n = _shape2("b", b)[0]
    kb = -(-k // 128)
    ld_a, ld_b = _matrix("a", a, index, shape, ta), _matrix("b", b, index, (n, k), tb)
    sa = _whole("a_scale", a_scale, index, (rows, kb), torch.float32)
    sb = _whole("b_scale", b_scale, index, (-(-n // 128), kb), torch.float32)
    if out is None:
        out, ld_out = torch.empty((rows, n), dtype=out_dtype, device=a.device), n
    else:
        ld_out = _matrix("out", out, index, (rows, n), out_dtype)
    args = MoeFfnFp8MatmulArgs(rows, n, k, _FP8[ta], _FP8[tb], _TYPES[out_dtype], a.data_ptr(), ld_a, sa, b.data_ptr(),
                               ld_b, sb, out.data_ptr(), ld_out)
    rc = _lib.load().moe_ffn_fp8_matmul(ctypes.byref(args), _raw_stream(index))
    if rc != 0:
        _raise(rc)
    return out


def dense_status(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Device status bits that the dense sublayer's kernels set on the current device (the stream's)
    since the last call, after waiting for the stream; then cleared."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dense_status()
    rc = _lib.load().moe_ffn_dense_status(_raw_stream(torch.cuda.current_device()))
    if rc < 0:
        _raise(rc)
    return rc
