"""fp8_matmul and fp8_quantise on the GPU against plain 64-bit arithmetic.

Tolerances, fixed by arithmetic.  fp8_matmul: the codes' products are exact in f32; a block's 128 are summed
in 4 steps of 32, each off by at most 2^-23 of the magnitudes' sum for the running sum and as much for the
products' alignment; the scales' product and the f32 multiply-adds over the blocks add 2^-24 of it each.  So
the sum over KB blocks is off by at most (8 + 8 + KB) 2^-23 M, M the sum of the magnitudes of all terms, and
the stored value by half a step of its type more.  fp8_quantise: the scale is one correctly rounded division
(2^-24); a code is the nearest to x * (1 / scale), whose reciprocal and product are rounded in f32 (2^-24
each): away from the border between two codes by 2^-23, the code is the one nearest to x / scale."""
import pytest
import torch

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2


def half_step(dtype, v):
    f = torch.finfo(dtype)
    return f.eps / 2 * v.abs() + f.smallest_normal * f.eps / 2


def operand(rows, k, tall, dtype, gen, pad=0):
    """Random codes over the whole finite range of the type, and random scales (positive and negative)."""
    v = torch.randn(rows, k + pad, generator=gen, device="cuda") * torch.exp2(
        torch.randint(-6, 7, (rows, k + pad), generator=gen, device="cuda").float())
    s = torch.randn(-(-rows // tall), -(-k // 128), generator=gen, device="cuda") * 0.1
    return v.to(dtype)[:, :k], s


def wide(q, s, tall):
    rows, k = q.shape
    return q.double() * s.double().repeat_interleave(tall, 0)[:rows].repeat_interleave(128, 1)[:, :k]


def check(a, sa, b, sb, out):
    da, db = wide(a, sa, 1), wide(b, sb, 128)
    ref, mag = da @ db.T, da.abs() @ db.abs().T
    tol = half_step(out.dtype, ref) + (16 + sa.shape[1]) * 2.0 ** -23 * mag
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), (float((err - tol).max()), float((err / tol).max()))


SIZES = [(1, 1, 16), (1, 129, 128), (2, 64, 144), (3, 1000, 256), (4, 4096, 4096), (5, 127, 384), (16, 200, 1040),
         (33, 1031, 2000), (128, 128, 128), (129, 257, 512), (200, 77, 4112), (300, 520, 272), (1000, 640, 1024),
         (1, 2048, 8192), (64, 8192, 512), (2100, 4000, 272), (1033, 2055, 640), (4096, 1031, 144)]


@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("ta,tb,out", [(E4, E4, BF16), (E5, E4, F32), (E4, E5, F16), (E5, E5, F32), (E4, E4, F32)])
def test_matmul(cuda_lib, rows, n, k, ta, tb, out):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(rows + n + k)
    a, sa = operand(rows, k, 1, ta, gen, pad=16 * (rows % 2))
    b, sb = operand(n, k, 128, tb, gen, pad=32 * (n % 2))
    if out == F16:
        sa, sb = sa * 2.0 ** -6, sb * 2.0 ** -6  # f16 results stay finite
    y = m.fp8_matmul(a, sa, b, sb, out_dtype=out)
    check(a, sa, b, sb, y)
    assert torch.equal(m.fp8_matmul(a, sa, b, sb, out_dtype=out), y)
    assert m.dense_status() == 0


def test_matmul_full_size(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(1)
    a, sa = m.fp8_quantise(torch.randn(4096, 4096, generator=gen, device="cuda").to(BF16))
    b, sb = m.fp8_quantise(torch.randn(4096, 4096, generator=gen, device="cuda").to(BF16), block_rows=128)
    check(a, sa, b, sb, m.fp8_matmul(a, sa, b, sb))


def test_exact_small_integers(cuda_lib):
    # codes and scales whose products and sums are all exact in f32: the result has every bit right
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(2)
    for rows, n, k in ((3, 300, 640), (260, 140, 400)):
        a = torch.randint(-4, 5, (rows, k), generator=gen, device="cuda").float().to(E4)
        b = torch.randint(-4, 5, (n, k), generator=gen, device="cuda").float().to(E5)
        sa = torch.exp2(torch.randint(-2, 3, (rows, -(-k // 128)), generator=gen, device="cuda").float())
        sb = torch.exp2(torch.randint(-2, 3, (-(-n // 128), -(-k // 128)), generator=gen, device="cuda").float())
        assert torch.equal(m.fp8_matmul(a, sa, b, sb, out_dtype=F32).double(), wide(a, sa, 1) @ wide(b, sb, 128).T)


def test_not_finite_stays_in_its_row_and_column(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(3)
    for rows in (4, 40):
        a, sa = operand(rows, 272, 1, E4, gen)
        b, sb = operand(300, 272, 128, E4, gen)
        clean = m.fp8_matmul(a, sa, b, sb, out_dtype=F32)
        sa[1, 2] = float("nan")
        b.view(torch.uint8)[5, 7] = 0x7F  # a NaN code
        y = m.fp8_matmul(a, sa, b, sb, out_dtype=F32)
        assert y[1].isnan().all() and y[:, 5].isnan().all()
        keep_r = [i for i in range(rows) if i != 1]
        keep_c = [i for i in range(300) if i != 5]
        assert torch.equal(y[keep_r][:, keep_c], clean[keep_r][:, keep_c])


def test_matmul_into_a_part_of_a_tensor(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(4)
    for rows in (2, 70):
        for n, pad in ((131, 5), (136, 8)):
            a, sa = operand(rows, 256, 1, E4, gen)
            b, sb = operand(n, 256, 128, E4, gen)
            big = torch.full((rows + 60, n + pad), 3.0, device="cuda", dtype=BF16)
            y = m.fp8_matmul(a, sa, b, sb, out=big[:rows, :n])
            check(a, sa, b, sb, y)
            assert (big[rows:] == 3).all() and (big[:, n:] == 3).all()


LIMITS = {E4: (448.0, 3, -6), E5: (57344.0, 2, -14)}


def check_quantised(x, tall, pow2, dtype, q, s):
    most, bits, low = LIMITS[dtype]
    rows, k = x.shape
    rb, kb = -(-rows // tall), -(-k // 128)
    full = torch.zeros(rb * tall, kb * 128, device="cuda", dtype=torch.float64)
    full[:rows, :k] = x.double()
    amax = full.view(rb, tall, kb, 128).abs().amax(dim=(1, 3))
    ref = torch.where(amax == 0, torch.ones_like(amax), (amax / most).clamp_min(2.0 ** -126))
    if pow2:
        e = torch.ceil(torch.log2(ref))
        e = torch.where(torch.exp2(e - 1) >= ref, e - 1, e)
        assert torch.equal(s.double(), torch.exp2(e))
    else:
        assert ((s.double() - ref).abs() <= 2.0 ** -24 * ref).all()
    v = x.double() / s.double().repeat_interleave(tall, 0)[:rows].repeat_interleave(128, 1)[:, :k]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - bits)
    err = (q.double() - v).abs()
    assert (err <= step / 2 + 2.0 ** -23 * v.abs()).all()
    # where v is clear of the border between two codes, the code is the nearest one
    near = (torch.round(v / step) * step).clamp(-most, most)
    clear = ((v / step - torch.floor(v / step) - 0.5).abs() * step) > 2.0 ** -23 * v.abs()
    assert torch.equal(q.double()[clear], near[clear])


@pytest.mark.parametrize("tall", [1, 128])
@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("xt,dtype", [(F32, E4), (BF16, E4), (F16, E5), (F32, E5)])
@pytest.mark.parametrize("rows,k", [(1, 1), (1, 4096), (3, 130), (129, 256), (130, 1000), (257, 77), (700, 2064)])
def test_quantise(cuda_lib, rows, k, tall, pow2, xt, dtype):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(rows * 7 + k)
    x = (torch.randn(rows, k + 3 * (k % 2), generator=gen, device="cuda")
         * torch.exp(torch.randn(rows, 1, generator=gen, device="cuda"))).to(xt)[:, :k]
    q, s = m.fp8_quantise(x, block_rows=tall, pow2_scales=pow2, dtype=dtype)
    assert q.dtype == dtype and q.shape == x.shape
    check_quantised(x, tall, pow2, dtype, q, s)


@pytest.mark.parametrize("tall", [1, 128])
def test_quantise_edges(cuda_lib, tall):
    import deepseek_v4_moe_gb300 as m
    x = torch.randn(256, 640, device="cuda", generator=torch.Generator(device="cuda").manual_seed(6))
    x[:, 128:256] = 0                        # blocks of zeros
    x[:, 256:384] *= 1e-38                   # subnormal magnitudes
    x[:, 384] = float("nan")
    x[:128, 512] = float("inf")
    q, s = m.fp8_quantise(x, block_rows=tall)
    assert (s[:, 1] == 1).all() and (q[:, 128:256].double() == 0).all()
    assert (s[:, 2] >= 2.0 ** -126).all()
    assert s[:, 3].isnan().all() and q[:, 384:512].double().isnan().all()
    top = 128 if tall == 1 else 1
    assert (s[:top, 4] == float("inf")).all() and s[top:, 4].isfinite().all()
    check_quantised(x[:, :256].contiguous(), tall, False, E4, q[:, :256], s[:, :2].contiguous())
    # largest values that are a power of two times the largest code: the scale is exact either way
    y = torch.full((128, 128), 0.875, device="cuda")
    for pow2 in (False, True):
        q, s = m.fp8_quantise(y, block_rows=tall, pow2_scales=pow2)
        assert (s == 2.0 ** -9).all() and (q.double() == 448).all()


def test_another_stream_and_a_graph(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(90, 528, generator=gen, device="cuda").to(BF16)
    w = torch.randn(300, 528, generator=gen, device="cuda").to(BF16)
    b, sb = m.fp8_quantise(w, block_rows=128)

    def step(stream=None):
        a, sa = m.fp8_quantise(x, stream=stream)
        return a, sa, m.fp8_matmul(a, sa, b, sb, stream=stream)

    first = step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    second = step(st)
    st.synchronize()
    assert all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(first, second))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, sa, y = step()
    x.copy_(torch.randn(90, 528, generator=gen, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    check_quantised(x, 1, False, E4, a, sa)
    check(a, sa, b, sb, y)


def test_a_wait_that_runs_out_is_reported(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(9)
    for rows, n, k in ((200, 256, 512), (4096, 4096, 1024)):  # single CTAs, and pairs
        a, sa = operand(rows, k, 1, E4, gen)
        b, sb = operand(n, k, 128, E4, gen)
        good = m.fp8_matmul(a, sa, b, sb)
        assert m.dense_status() == 0
        assert cuda_lib.moe_ffn_dense_fault_injection(1, 20000) == 0
        try:
            m.fp8_matmul(a, sa, b, sb)
            assert m.dense_status() == 8
        finally:
            cuda_lib.moe_ffn_dense_fault_injection(0, 0)
        assert torch.equal(m.fp8_matmul(a, sa, b, sb), good)
        assert m.dense_status() == 0


def test_refusals(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(10)
    a, sa = operand(5, 256, 1, E4, gen)
    b, sb = operand(200, 256, 128, E4, gen)
    for bad in (lambda: m.fp8_matmul(a.float(), sa, b, sb), lambda: m.fp8_matmul(a, sa[:, :1], b, sb),
                lambda: m.fp8_matmul(a, sa.double(), b, sb), lambda: m.fp8_matmul(a, sa, b[:, :128], sb),
                lambda: m.fp8_matmul(a, sa, b, sb[:1]), lambda: m.fp8_matmul(a, sa, b, sb, out_dtype=torch.float64),
                lambda: m.fp8_matmul(a.cpu(), sa, b, sb), lambda: m.fp8_quantise(sa.long()),
                lambda: m.fp8_quantise(sa, block_rows=64), lambda: m.fp8_quantise(sa, dtype=torch.int8),
                lambda: m.fp8_quantise(sa.cpu())):
        with pytest.raises(ValueError):
            bad()
    x = torch.zeros(5, 40, device="cuda").to(E4)
    for code, bad in ((-4, lambda: m.fp8_matmul(a[:0], sa[:0], b, sb)), (-4, lambda: m.fp8_quantise(sa[:0])),
                      (-2, lambda: m.fp8_matmul(x, sa[:, :1].contiguous(), x, torch.ones(1, 1, device="cuda"))),
                      (-2, lambda: m.fp8_matmul(a[:, :40], sa[:, :1].contiguous(), b[:, :40], sb[:, :1].contiguous()))):
        with pytest.raises(m.MoeFFNError) as e:
            bad()
        assert e.value.code == code
