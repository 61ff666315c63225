"""fp8_matmul with scales whose product leaves f32's normal range, though the results do not.

Tolerance: that of the product's own tests, (16 + KB) 2^-23 of the terms' magnitudes and the stored value's half
step, as a term is still rounded twice (its sum times one scale; times the other and added).  Sums below the
normal range are rounded to multiples of 2^-149: at most half of one in each of the 8 KB steps of a few rows'
kernel and the 40 in which its partial sums meet."""
import pytest
import torch

import test_gpu_fp8 as t8

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2

# few rows with one column and with four a warp; tiles of 32 to 256 columns by one CTA, pairs and clusters
SIZES = [(1, 300, 640), (3, 300, 272), (2, 10000, 272), (47, 133, 160), (8, 4935, 176), (17, 20, 2944), (539, 3903, 1152),
         (2619, 1376, 2208), (4958, 200, 2656), (1033, 2055, 640)]


def operands(rows, n, k, kind, gen):
    """Codes and scales, E5M2: `small` and `large` products in every block; `rows` and `columns` of them beside
    ordinary ones; `apart`: the products of the scales are past f32's range where every product of codes is 0."""
    kb, nb = -(-k // 128), -(-n // 128)

    def rnd(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    a, b = rnd(rows, k) * 4, rnd(n, k) * 4
    sa, sb = rnd(rows, kb), rnd(nb, kb)
    sa, sb = sa.sign() * (0.5 + sa.abs()), sb.sign() * (0.5 + sb.abs())
    i, j = torch.arange(rows, device="cuda")[:, None], torch.arange(nb, device="cuda")[:, None]
    if kind == "small":
        a, b, sa, sb = a * 2.0 ** 10, b * 2.0 ** 10, sa * 2.0 ** -80, sb * 2.0 ** -58
    elif kind == "large":
        a, b, sa, sb = a * 2.0 ** -14, b * 2.0 ** -14, sa * 2.0 ** 80, sb * 2.0 ** 54
    elif kind in ("rows, small", "rows, large"):
        e = torch.where(i % 3 == 0, -100.0 if kind == "rows, small" else 100.0, 0.0)
        a = a * torch.where(e < 0, 2.0 ** 10, torch.where(e > 0, 2.0 ** -14, 1.0))
        b = b * 2.0 ** (10 if kind == "rows, small" else -10)
        sa, sb = sa * torch.exp2(e), sb * 2.0 ** (-40 if kind == "rows, small" else 32)
    elif kind == "columns":
        e = torch.tensor([-62.0, 0.0, 50.0], device="cuda")[j % 3]
        of = e.repeat_interleave(128, 0)[:n]
        b = b * torch.where(of < 0, 2.0 ** 10, torch.where(of > 0, 2.0 ** -14, 1.0))
        sa, sb = sa * torch.where(i % 2 == 0, 2.0 ** -80, 2.0 ** 82), sb * torch.exp2(e)
        a = torch.where(i % 2 == 0, a * 2.0 ** 10, a * 2.0 ** -14)
    else:
        odd = torch.arange(k, device="cuda") % 2 == 1
        a, b = torch.where(odd, a, 0.0), torch.where(odd, 0.0, b)
        sa, sb = sa * 2.0 ** 100, sb * 2.0 ** 90
        sa[:, -1], sb[:, -1] = 0.25, 0.5
        a[:, 128 * (kb - 1):] = 2.0
    return a.to(E5), sa, b.to(E5), sb


@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("kind", ["small", "large", "rows, small", "rows, large", "columns", "apart"])
@pytest.mark.parametrize("out", [F32, BF16])
def test_products_of_scales_out_of_range(cuda_lib, rows, n, k, kind, out):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(rows + n + k)
    a, sa, b, sb = operands(rows, n, k, kind, gen)
    product = sa.double()[:, None, :] * sb.double()[None]
    lost = (product.abs() < 2.0 ** -126) | (product.abs() >= 2.0 ** 128)
    assert lost.any()
    da, db = t8.wide(a, sa, 1), t8.wide(b, sb, 128)
    ref, mag = da @ db.T, da.abs() @ db.abs().T
    assert float(mag.max()) < 2.0 ** 126
    y = m.fp8_matmul(a, sa, b, sb, out_dtype=out)
    tol = t8.half_step(out, ref) + (16 + sa.shape[1]) * 2.0 ** -23 * mag + (8 * sa.shape[1] + 40) * 2.0 ** -150
    err = (y.double() - ref).abs()
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    assert torch.equal(m.fp8_matmul(a, sa, b, sb, out_dtype=out), y)
    assert m.dense_status() == 0


def test_scales_that_the_quantiser_makes(cuda_lib):
    """Rows of 1e-24 and of 1e22, quantised: their products are normal f32 values."""
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(1)
    for rows in (2, 40):
        for size in (1e-17, 1e18):
            x = torch.randn(rows, 512, generator=gen, device="cuda") * size
            w = torch.randn(300, 512, generator=gen, device="cuda") * size
            a, sa = m.fp8_quantise(x, dtype=E5)
            b, sb = m.fp8_quantise(w, block_rows=128, dtype=E5)
            t8.check(a, sa, b, sb, m.fp8_matmul(a, sa, b, sb, out_dtype=F32))
    # a block of a whose only value meets zeros: 0, whatever the scales
    a = torch.zeros(3, 128, device="cuda")
    a[:, 5] = 1e25
    b = torch.full((200, 128), 1e25, device="cuda")
    b[:, 5] = 0
    for rows in (1, 3):
        y = m.fp8_matmul(*m.fp8_quantise(a[:rows].contiguous()), *m.fp8_quantise(b, block_rows=128), out_dtype=F32)
        assert (y == 0).all()
    y = m.fp8_matmul(*m.fp8_quantise(a.repeat(20, 1)), *m.fp8_quantise(b, block_rows=128), out_dtype=F32)
    assert (y == 0).all()
