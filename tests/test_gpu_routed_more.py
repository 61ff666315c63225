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


@pytest.mark.parametrize("power,inverse", [(-100, 100), (100, -100), (126, -110)])
def test_tokens_of_any_magnitude(power, inverse):
    """Tokens times a power of two, up to the end of bf16, and the scales of gate and up times another."""
    x, router, ws, _, _ = tr.layer(6, 256, 160, 12, 0, 4, 64, False, BF16, False, False)
    x = torch.where(x.abs() < 2.0 ** -8, 2.0 ** -8, x).clamp(-1.5, 1.5)  # (no value leaves the normal numbers)
    router, bias = torch.zeros_like(router), torch.arange(12, device="cuda") / 12
    ws2 = [w._replace(scales=w.scales * 2.0 ** inverse) for w in ws[:2]] + [ws[2]]
    got = m.routed_ffn(x * 2.0 ** power, router, *ws2, 3, bias=bias)
    if power + inverse == 0:  # every step is exact up to the powers
        assert all(torch.equal(a, b) for a, b in zip(got, m.routed_ffn(x, router, *ws, 3, bias=bias)))
    tr.check(got, x * 2.0 ** power, router, ws2, 3, None, "silu", bias)
