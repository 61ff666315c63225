"""gated_quantise where the sigmoid is small: its float32 arithmetic against 64 bits."""
import pytest
import torch

import deepseek_v4_moe_gb300 as m
from test_gpu_fp8_out import check_codes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lo,hi", [(-87.0, -84.0), (-84.0, -40.0), (-40.0, -10.0), (-10.0, 10.0), (10.0, 1000.0)])
@pytest.mark.parametrize("inter", [1024, 1001])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_silu_far_out(lo, hi, inter, dtype):
    """The sigmoid off by 2^-21 at most (of normal numbers: not below exp(-87)), two products and the block's scale by half a
    unit of 2^-23 each: below 2^-20."""
    g = torch.Generator("cuda").manual_seed(inter)
    gate = (torch.rand(40, inter, generator=g, device="cuda") * (hi - lo) + lo).to(dtype)
    # (up brings the products back from exp's end, so that no scale is cut at its least value, 2^-126)
    up = (torch.randn(40, inter, generator=g, device="cuda") * (2.0 ** 14 if dtype == torch.float16 else 2.0 ** 40)).to(dtype)
    up = torch.where(torch.isfinite(up), up, 1.0)
    codes, scales = m.gated_quantise(gate, up)
    a = gate.double()
    check_codes(codes, scales, a * torch.sigmoid(a) * up.double(), "e4m3", False, 2.0 ** -20)
