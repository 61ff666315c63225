"""Python face of the dense feed-forward sublayer (plain residual stream) over the C entry points of
include/moe_ffn.h; the checks and the marshalling are in the compiled binding (csrc/binding.cpp).

Every function enqueues on ``stream`` (default: the tensors' device's current stream) and returns
device tensors without waiting.  Outputs and workspaces that a call allocates belong to that stream;
inputs that belong to another one stay with the caller until the call's kernels have run.
Gradients come from explicit ``*_backward`` calls; nothing is recorded for autograd, also where an argument
requires a gradient.  Tensors given for a call to write into count as changed in place.  Rows may be
strided (``stride(-1) == 1``) but not lie in one another, as an expanded tensor's do; weights and gates are
contiguous.  Refused arguments raise
``ValueError`` (types, shapes), ``TypeError`` (no tensor) or ``MoeFFNError`` with the library's code.
"""
from __future__ import annotations

import importlib
from typing import Optional

import torch

from . import _lib
from ._lib import ACTIVATIONS
from .api import MoeFFNError

_n = None  # the binding, once loaded


def _native():
    global _n
    if _n is None:
        from . import build
        _lib.load()  # builds what is missing
        if not build.native_fits():
            raise RuntimeError(f"{build.NATIVE} is missing or was built for another PyTorch, Python or interface, and "
                               f"was not built anew") from _lib.build_error
        n = importlib.import_module("._native", __package__)
        n.set_error(MoeFFNError)
        _n = n
    return _n


def _on(t: torch.Tensor, stream: torch.cuda.Stream):
    """The context to run a call on tensor t on another stream in."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"a torch.Tensor is needed, got {type(t).__name__}")
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
    return torch.cuda.stream(stream)


def _activation(name: str) -> int:
    if name not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[name]


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
    if stream is not None:
        with _on(state, stream):
            return (_n or _native()).block_norm(state, f, norm_f, gate, residual_scale, norm_next, eps, block_dtype, out, y)
    return (_n or _native()).block_norm(state, f, norm_f, gate, residual_scale, norm_next, eps, block_dtype, out, y)


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
    if stream is not None:
        with _on(out, stream):
            return (_n or _native()).block_norm_backward(out, f, norm_f, gate, residual_scale, norm_next, eps, d_out, d_y)
    return (_n or _native()).block_norm_backward(out, f, norm_f, gate, residual_scale, norm_next, eps, d_out, d_y)


def gated_ffn(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
              activation: str = "silu", save: bool = False, out: Optional[torch.Tensor] = None,
              stream: Optional[torch.cuda.Stream] = None):
    """The gated feed-forward block: y = (act(x w_gate^T) * (x w_up^T)) w_down^T.

    ``x`` [rows, hidden] bfloat16 or float16; ``w_gate``, ``w_up`` [inter, hidden] and ``w_down``
    [hidden, inter] of its type; hidden and inter multiples of 8, every tensor 16-byte aligned and row
    strides multiples of 8.  ``activation``: "silu" or "gelu"
    (tanh form).  Sums are float32; the activated product is rounded to x's type before the down projection (in
    float16 past 65504 to infinity), while the routed block keeps its own in two parts.  Returns y [rows, hidden]; with ``save`` also the pair (g, u) of projections
    [rows, inter] that :func:`gated_ffn_backward` takes.
    """
    if stream is not None:
        with _on(x, stream):
            return (_n or _native()).gated_ffn(x, w_gate, w_up, w_down, _activation(activation), save, out)
    return (_n or _native()).gated_ffn(x, w_gate, w_up, w_down, _activation(activation), save, out)


def gated_ffn_backward(x: torch.Tensor, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, saved,
                       d_y: torch.Tensor, activation: str = "silu", need_x: bool = True, need_weights: bool = True,
                       stream: Optional[torch.cuda.Stream] = None) -> dict:
    """Gradients of :func:`gated_ffn` from what it saved: a dict of d_x, d_w_gate, d_w_up and d_w_down
    (of the inputs' type), without d_x or the weights' where they are not needed.  The gradients of the two
    projections and the activated product are rounded to that type on the way."""
    if stream is not None:
        with _on(x, stream):
            return (_n or _native()).gated_ffn_backward(x, w_gate, w_up, w_down, saved[0], saved[1], d_y,
                                                        _activation(activation), need_x, need_weights)
    return (_n or _native()).gated_ffn_backward(x, w_gate, w_up, w_down, saved[0], saved[1], d_y,
                                                _activation(activation), need_x, need_weights)


def fp8_quantise(x: torch.Tensor, block_rows: int = 1, pow2_scales: bool = False,
                 dtype: torch.dtype = torch.float8_e4m3fn, stream: Optional[torch.cuda.Stream] = None):
    """Makes an operand of :func:`fp8_matmul`: (codes [rows, k] of ``dtype``, float32 scales
    [ceil(rows / block_rows), ceil(k / 128)]).

    ``x`` [rows, k] float32, bfloat16 or float16.  ``block_rows`` 1 (activations) or 128 (weights).  A
    block's scale is its largest magnitude over the largest code, 1 for zeros, at least 2^-126, with
    ``pow2_scales`` rounded up to a power of two; a code is the quotient x / scale rounded to nearest even.
    """
    if stream is not None:
        with _on(x, stream):
            return (_n or _native()).fp8_quantise(x, block_rows, pow2_scales, dtype)
    return (_n or _native()).fp8_quantise(x, block_rows, pow2_scales, dtype)


def fp8_matmul(a: torch.Tensor, a_scale: torch.Tensor, b: torch.Tensor, b_scale: torch.Tensor,
               out_dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """a b^T of FP8 operands with float32 scales for blocks of 128: ``a`` [rows, k] with ``a_scale``
    [rows, ceil(k / 128)], ``b`` [n, k] with ``b_scale`` [ceil(n / 128), ceil(k / 128)] (see
    :func:`fp8_quantise`; each float8_e4m3fn or float8_e5m2), k and both row strides multiples of 16, both
    16-byte aligned.  Sums are float32; the
    result is ``out_dtype``: float32, bfloat16 or float16.
    """
    if stream is not None:
        with _on(a, stream):
            return (_n or _native()).fp8_matmul(a, a_scale, b, b_scale, out_dtype, out)
    return (_n or _native()).fp8_matmul(a, a_scale, b, b_scale, out_dtype, out)


def dense_status(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Device status bits that the dense sublayer's kernels set on the current device (the stream's)
    since the last call, after waiting for the stream; then cleared."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return dense_status()
    lib = _lib.load()
    rc = lib.moe_ffn_dense_status(torch.cuda.current_stream().cuda_stream)
    if rc < 0:
        raise MoeFFNError(rc, lib.moe_ffn_last_error(None).decode())
    return rc
