"""Python face of the products with 4-bit weights and of the routed layer without a handle, for serving a few tokens,
over the C entry points of include/moe_ffn.h.

Streams, outputs, strides and refusals are as in :mod:`.dense`: every function enqueues on ``stream`` (default: the
tensors' device's current stream) and returns device tensors without waiting; nothing is recorded for autograd.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple, Union

import torch

from . import dense
from ._lib import SCORES
from .dense import _activation, _native, _on


class Int4(NamedTuple):
    """Weights [..., n, k] in 4 bits: w = (code - zero) * scale, a scale (and zero point) for each ``group`` columns.

    ``codes`` uint8 [..., n, k / 2], the even column in the low half of a byte; ``scales`` bfloat16 or float16
    [..., n, ceil(k / group)]; ``zeros`` uint8 of that shape (the low four bits of each), or None for 8; ``group`` 32, 64
    or 128.  All contiguous and 16-byte aligned; k a multiple of 32.
    """
    codes: torch.Tensor
    scales: torch.Tensor
    zeros: Optional[torch.Tensor] = None
    group: int = 128


Weights = Union[torch.Tensor, Int4]


def int4_quantise(w: torch.Tensor, group: int = 128, zero_points: bool = False,
                  scale_dtype: Optional[torch.dtype] = None, stream: Optional[torch.cuda.Stream] = None) -> Int4:
    """Weights [..., n, k] float32, bfloat16 or float16 in 4 bits.

    Symmetric: scale = max|w| / 7 of a group, codes 1..15 around 8.  With ``zero_points``: scale = (max(w, 0) -
    min(w, 0)) / 15, codes 0..15 around zero = -min(w, 0) / scale.  Scales are rounded to ``scale_dtype`` (default: w's
    type, bfloat16 for float32), are 1 for zeros and at least its smallest normal value; codes are the quotients by the
    scale as stored, rounded to nearest even.
    """
    if stream is not None:
        with _on(w, stream):
            return Int4(*(dense._n or _native()).int4_quantise(w, group, zero_points, scale_dtype))
    return Int4(*(dense._n or _native()).int4_quantise(w, group, zero_points, scale_dtype))


def int4_widen(w: Int4, out: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The values of 4-bit weights [..., n, k], rounded to the scales' type: for a prompt, whose products
    :func:`gated_ffn` makes."""
    if stream is not None:
        with _on(w[0], stream):
            return (dense._n or _native()).int4_widen(w, out)
    return (dense._n or _native()).int4_widen(w, out)


def int4_matmul(x: torch.Tensor, w: Int4, out: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """x w^T for a few rows: ``x`` [rows, k] bfloat16 or float16 (16-byte aligned, row strides multiples of 8), ``w``
    [n, k] in 4 bits with scales of x's type.  Each group's products are summed in float32 and multiplied by its scale
    there; the result [rows, n] is of x's type.  Made for up to 32 rows; more are taken 32 at a time.

    Large products and those of more rows take x in FP8 planes: exact down to 2^-14 of a row's largest magnitude (float16:
    2^-16), off by at most 2^-22 (2^-27) of it below that.  A row that is not finite gives no finite result: NaN there,
    infinities among them elsewhere.
    """
    if stream is not None:
        with _on(x, stream):
            return (dense._n or _native()).int4_matmul(x, w, out)
    return (dense._n or _native()).int4_matmul(x, w, out)


def routed_ffn(x: torch.Tensor, w_router: torch.Tensor, w_gate: Weights, w_up: Weights, w_down: Weights, top_k: int, *,
               bias: Optional[torch.Tensor] = None, score: str = "sigmoid", normalise: bool = True,
               route_scale: float = 1.0, shared: Optional[Tuple[Weights, Weights, Weights]] = None,
               activation: str = "silu", out: Optional[torch.Tensor] = None,
               stream: Optional[torch.cuda.Stream] = None):
    """A whole mixture-of-experts layer for up to 32 tokens, without a handle or hyper-connections.

        l = x w_router^T;  s = sigmoid(l) or softmax(l)
        the top_k experts by s + bias, ties to the lower index;  weight = route_scale * s / (sum of the chosen s)
        y = sum of weight * expert(x) + sum of the shared experts' (x), each a gated block as :func:`gated_ffn`'s

    ``x`` [rows, hidden] bfloat16 or float16; ``w_router`` [experts, hidden] float32 or of x's type; ``bias`` float32
    [experts]; ``w_gate``, ``w_up`` [experts, inter, hidden] and ``w_down`` [experts, hidden, inter], tensors of x's type
    or all :class:`Int4` of one group; ``shared``: the same three of the shared experts, [inter, hidden] for one or
    [count, inter, hidden].  hidden and inter are multiples of 8 (32 with Int4).  Without ``normalise`` the weight is
    route_scale * s.  The hidden values go into the down projection as two numbers of x's type; with 4-bit experts x goes
    through planes as :func:`int4_matmul`'s does and the hidden values through three, off by at most 2^-14 of a value or
    2^-27 of the token's largest.  What is not finite in a token or an expert reaches that token, or the tokens that
    have chosen the expert, alone.  Returns (y [rows, hidden], indices int32 [rows, top_k], weights float32 [rows, top_k]).
    """
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}")
    args = (x, w_router, w_gate, w_up, w_down, top_k, bias, SCORES[score], normalise, route_scale,
            tuple(shared) if shared is not None else None, _activation(activation), out)
    if stream is not None:
        with _on(x, stream):
            return (dense._n or _native()).routed_ffn(*args)
    return (dense._n or _native()).routed_ffn(*args)
