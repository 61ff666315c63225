"""fp8_quantise's codes are those of the quotients x / scale: each the correctly rounded f32 quotient, rounded to the
code's type, bit for bit what the CPU's division and conversion give."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
MOST = {E4: 448.0, E5: 57344.0}


def want(x, s, tall, dtype):
    rows, k = x.shape
    x, s = x.cpu().float(), s.cpu().repeat_interleave(tall, 0)[:rows].repeat_interleave(128, 1)[:, :k]
    return (x / s).clamp(-MOST[dtype], MOST[dtype]).to(dtype)


def same(q, ref):
    q, ref = q.cpu().view(torch.uint8), ref.view(torch.uint8)
    assert torch.equal(q, ref), f"{int((q != ref).sum())} of {q.numel()} codes"


@pytest.mark.parametrize("xt", [F32, BF16, F16])
@pytest.mark.parametrize("dtype", [E4, E5])
@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("rows,k", [(1, 77), (257, 2064), (2000, 1003), (1024, 4096)])
def test_codes_of_the_quotients(cuda_lib, xt, dtype, tall, pow2, rows, k):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(rows + k)
    x = (torch.randn(rows, k, generator=gen, device="cuda")
         * torch.exp(torch.randn(rows, 1, generator=gen, device="cuda"))).to(xt)
    x[::3, ::5] *= 0  # zeros of both signs
    q, s = m.fp8_quantise(x, block_rows=tall, pow2_scales=pow2, dtype=dtype)
    same(q, want(x, s, tall, dtype))


@pytest.mark.parametrize("dtype", [E4, E5])
def test_values_next_to_the_border_between_two_codes(cuda_lib, dtype):
    """A block's largest value sets its scale; the others are the f32 values at and around the border between two
    codes times that scale."""
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.arange(0, 0x7e if dtype == E4 else 0x7b, dtype=torch.uint8).view(dtype).double().cuda()
    border = (codes[1:] + codes[:-1]) / 2
    rows = 4000
    top = (1 + torch.rand(rows, 1, generator=gen, device="cuda")) * 2.0 ** torch.randint(-30, 30, (rows, 1), generator=gen, device="cuda")
    s_want = (top.cpu() / torch.tensor(MOST[dtype])).cuda()  # (PyTorch's GPU division by a number is by its reciprocal)
    scale = s_want.double()
    at = border[torch.randint(0, len(border), (rows, 127), generator=gen, device="cuda")]
    x = (at * scale).float()
    x = torch.nextafter(x, x * torch.randint(0, 3, x.shape, generator=gen, device="cuda"))  # below, at or above
    x = torch.cat([top, x * torch.where(torch.rand(x.shape, generator=gen, device="cuda") < 0.5, 1.0, -1.0)], 1)
    q, s = m.fp8_quantise(x, dtype=dtype)
    assert torch.equal(s, s_want)
    same(q, want(x, s, 1, dtype))
