"""gated_ffn_backward at gates as far out as the type holds: the activation's derivative is 1 or 0 there."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("rows", [1, 9, 200])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gates_past_the_square_root_of_f32(cuda_lib, rows, name):
    # g = x, u = c x, dh = 1: dg = c x act'(g) and du = act(g), so d_x = dg + c du = 2 c x for positive x, 0 for
    # negative.  c is a power of two; dg and du are rounded to bf16 (2^-8 each), their sum once more.
    import deepseek_v4_moe_gb300 as m
    c = 2.0 ** -100
    eye = torch.eye(64, device="cuda", dtype=BF16)
    sizes = torch.tensor([1e14, 3e18, 5e19, 1e20, 1e26, 1e32, 3e38, 16.0], device="cuda")
    x = (sizes.repeat(rows, 8) * torch.where(torch.arange(64, device="cuda") < 32, 1.0, -1.0)).to(BF16)
    y, saved = m.gated_ffn(x, eye, (eye * c).to(BF16), eye, activation=name, save=True)
    assert torch.equal(saved[0], x)
    d = m.gated_ffn_backward(x, eye, (eye * c).to(BF16), eye, saved, torch.ones_like(x), activation=name,
                             need_weights=False)["d_x"].double()
    want = 2 * c * x.double().clamp_min(0)
    # at -16, exp(-16) = 1.2e-7 of silu is left: |act'| <= 2e-6
    tol = 3 * 2.0 ** -8 * want.abs() + 2 * c * x.double().abs() * torch.where(x.abs() < 20, 2e-6, 0.0)
    assert ((d - want).abs() <= tol).all(), (d[0], want[0])
