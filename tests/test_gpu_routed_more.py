"""The routed layer without a handle, further: the choice's place in shared memory, magnitudes at the types' ends, the
precision of the hidden values, weights that are not finite, and the choice of every token."""
import math

import pytest
import torch

import deepseek_v4_moe_gb300 as m
import test_gpu_int4 as t4
import test_gpu_routed as tr

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.mark.parametrize("bits,rows", [(16, 3), (16, 32), (4, 3), (4, 32)])
def test_the_choice_and_the_weights_share_shared_memory(bits, rows):
    """The most experts: their keys fill the place that weights are copied to next, in every kernel.  The same bits each
    time, and right."""
    x, router, ws, _, bias = tr.layer(rows, 288, 128, 512, 0, bits, 64, True, BF16, False, True)
    first = m.routed_ffn(x, router, *ws, 8, bias=bias)
    tr.check(first, x, router, ws, 8, None, "silu", bias)
    for _ in range(50):
        again = m.routed_ffn(x, router, *ws, 8, bias=bias)
        assert all(torch.equal(a, b) for a, b in zip(again, first))
