"""Tensors that a call writes into count as changed for autograd, which then refuses a gradient that would be
taken of the old values."""
import pytest
import torch

import test_gpu_fp8 as t8

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def test_outputs_given_by_the_caller_count_as_changed(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    h = 64
    w = torch.ones(h, device="cuda")
    eye = torch.eye(h, device="cuda", dtype=BF16)

    def given(dtype=BF16):
        return torch.full((5, h), 2.0, device="cuda", dtype=dtype)

    x, f = given(), given()
    gen = torch.Generator(device="cuda").manual_seed(0)
    a, sa = t8.operand(5, 128, 1, torch.float8_e4m3fn, gen)
    b, sb = t8.operand(h, 128, 128, torch.float8_e4m3fn, gen)
    for call in (lambda t: m.block_norm(x, f, out=t), lambda t: m.block_norm(t, f, out=t),
                 lambda t: m.block_norm(x, norm_next=w, y=t), lambda t: m.gated_ffn(x, eye, eye, eye, out=t),
                 lambda t: m.fp8_matmul(a, sa, b, sb, out=t)):
        t = given()
        v = torch.ones(5, h, device="cuda", dtype=BF16, requires_grad=True)
        loss = (t * v).sum()  # keeps t for v's gradient
        before = t._version
        call(t)
        assert t._version > before
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
    # inputs are not changed, and tensors of inference mode have no versions
    before = x._version, f._version
    m.block_norm(x, f)
    assert (x._version, f._version) == before
    with torch.inference_mode():
        t = given()
        m.block_norm(x, f, out=t)
        m.block_norm(t, f, out=t)
    m.block_norm(x, f, out=t)
    torch.cuda.synchronize()
