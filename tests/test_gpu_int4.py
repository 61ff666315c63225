"""Products with 4-bit weights, and making and widening them, against 64-bit arithmetic."""
import math

import pytest
import torch

import deepseek_v4_moe_gb300 as m

pytestmark = pytest.mark.gpu

LEAST = {torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -14}
# A group's sum: at most 8 accumulations of 16 products, whose alignment may lose a unit of 2^-23 each; then up to 64
# groups and 8 warps: below 2^7 units of 2^-23 of the sum of magnitudes.
SUM_SLACK = 2.0 ** -16


def values(w, group):
    codes, scales, zeros = w
    k = 2 * codes.shape[-1]
    at = torch.arange(k, device=codes.device)
    q = ((codes[..., at // 2].int() >> (4 * (at % 2)).int()) & 15).double()
    z = (zeros[..., at // group] & 15).double() if zeros is not None else 8
    return (q - z) * scales[..., at // group].double()


def make(shape, dtype, group, zeros, g):
    *lead, k = shape
    groups = -(-k // group)
    codes = torch.randint(0, 256, (*lead, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((torch.rand(*lead, groups, generator=g, device="cuda") + 0.5) * 0.25 * k ** -0.5).to(dtype)
    z = torch.randint(0, 16, (*lead, groups), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return m.Int4(codes, scales, z, group)


def check_product(y, x, w, first=0):
    v = values(w[:3], w.group)
    want, size = x.double() @ v.T, x.double().abs() @ v.abs().T
    room = torch.finfo(x.dtype).eps / 2 * want.abs() + SUM_SLACK * size
    if x.dtype == torch.float16:
        room = room + 2.0 ** -25
    assert y.dtype == x.dtype and y.shape == want.shape
    assert ((y.double() - want).abs() <= room * (1 + 2.0 ** -7)).all()


SIZES = [(1, 1, 32), (1, 16, 64), (2, 17, 96), (3, 100, 128), (7, 15, 160), (8, 31, 256), (9, 33, 288), (13, 1031, 2016),
         (16, 64, 512), (17, 130, 1024), (31, 128, 4096), (32, 257, 544), (33, 40, 320), (64, 200, 8192), (65, 513, 480),
         (1, 4096, 4096), (5, 10000, 256), (12, 20011, 64), (40, 9729, 128), (2, 3, 20000)]


@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("dtype,group,zeros", [(torch.bfloat16, 128, False), (torch.float16, 32, True),
                                               (torch.bfloat16, 64, True), (torch.float16, 128, True),
                                               (torch.bfloat16, 32, False)])
def test_int4_matmul(rows, n, k, dtype, group, zeros):
    g = torch.Generator("cuda").manual_seed(rows * 7919 + n * 31 + k)
    x = torch.randn(rows, k, generator=g, device="cuda").to(dtype)
    w = make((n, k), dtype, group, zeros, g)
    check_product(m.int4_matmul(x, w), x, w)


def test_every_code_column_and_zero_point():
    """One column at a time with a power of two: the result is the code less its zero point, exactly."""
    k = 512
    for group, zeros in ((32, True), (64, False), (128, True)):
        g = torch.Generator("cuda").manual_seed(group)
        w = make((40, k), torch.bfloat16, group, zeros, g)
        w = m.Int4(w.codes, torch.full_like(w.scales, 0.5), w.zeros, group)
        eye = 2 * torch.eye(k, device="cuda", dtype=torch.bfloat16)
        got = torch.cat([m.int4_matmul(eye[i:i + 13], w) for i in range(0, k, 13)])
        assert torch.equal(got.double(), 2 * values(w[:3], group).T)


def test_strided_rows_given_output_and_values_that_are_not_finite():
    g = torch.Generator("cuda").manual_seed(1)
    wide = torch.randn(11, 1000, generator=g, device="cuda").bfloat16()
    x = wide[:, 8:8 + 640]
    w = make((77, 640), torch.bfloat16, 128, True, g)
    out = torch.full((11, 100), 7.0, device="cuda", dtype=torch.bfloat16)
    version = out._version
    got = m.int4_matmul(x, w, out=out[:, 3:80])
    assert got.data_ptr() == out[:, 3:80].data_ptr() and out._version > version
    check_product(out[:, 3:80], x, w)
    assert (out[:, :3] == 7).all() and (out[:, 80:] == 7).all()
    # a row that is not finite leaves the others as they are
    bad = x.clone()
    bad[4, 100], bad[9, 3] = math.nan, math.inf
    y = m.int4_matmul(bad, w)
    keep = [i for i in range(11) if i not in (4, 9)]
    assert torch.equal(y[keep], got[keep]) and torch.isnan(y[4]).all() and not torch.isfinite(y[9]).any()


def test_the_same_bits_again_on_another_stream_and_replayed():
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(20, 2048, generator=g, device="cuda").half()
    w = make((3000, 2048), torch.float16, 64, False, g)
    first = m.int4_matmul(x, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = m.int4_matmul(x, w, stream=side)
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = m.int4_matmul(x, w)
    torch.cuda.synchronize()
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    # (not first / 2: half of an f16 below 2^-13 is rounded)
    assert torch.equal(first, again) and torch.equal(kept, m.int4_matmul(x, w)) and not torch.equal(kept, first)


def test_offsets_past_32_bits():
    """Codes of more than 2^32 bytes: the last rows' results."""
    n, k = 1048591, 8256
    codes = torch.zeros(n, k // 2, device="cuda", dtype=torch.uint8)
    assert codes.numel() > 2 ** 32
    g = torch.Generator("cuda").manual_seed(3)
    tail = make((37, k), torch.bfloat16, 128, True, g)
    codes[-37:] = tail.codes
    scales = torch.ones(n, tail.scales.shape[1], device="cuda", dtype=torch.bfloat16)
    zeros = torch.zeros(n, tail.scales.shape[1], device="cuda", dtype=torch.uint8)
    scales[-37:], zeros[-37:] = tail.scales, tail.zeros
    x = torch.randn(2, k, generator=g, device="cuda").bfloat16()
    y = m.int4_matmul(x, m.Int4(codes, scales, zeros, 128))
    assert (y[:, :-37] == 0).all()
    check_product(y[:, -37:], x, tail)


# ---- making and widening ----


def quantised(w, group, zero_points, dtype):
    """Codes, scales and zero points by their definition: quotients in 64 bits of numbers that 32 bits hold, rounded once."""
    *lead, k = w.shape
    v = torch.nn.functional.pad(w.double(), (0, -k % group)).unflatten(-1, (-1, group))
    lo, hi = v.amin(-1).clamp_max(0), v.amax(-1).clamp_min(0)
    f32 = lambda a: a.float().double()  # noqa: E731  the step's rounding
    s = f32(f32(hi - lo) / 15) if zero_points else f32(torch.maximum(hi, -lo) / 7)
    s = torch.where(s == 0, torch.ones_like(s), s.clamp_min(LEAST[dtype])).to(dtype)
    d = s.double()
    zero = torch.round(f32(-lo / d)).clamp(0, 15) if zero_points else torch.full_like(d, 8)
    q = (torch.round(f32(v / d[..., None])) + zero[..., None]).clamp(0 if zero_points else 1, 15)
    q = q.flatten(-2)[..., :k].to(torch.uint8)
    return q[..., ::2] | q[..., 1::2] << 4, s, zero.to(torch.uint8) if zero_points else None


@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (5, 128), (17, 160), (33, 2016), (257, 1024), (2, 3, 5, 64), (4, 100, 288)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("group,zero_points,scale_dtype", [(128, False, None), (32, True, torch.float16), (64, True, torch.bfloat16),
                                                           (64, False, torch.float16)])
def test_int4_quantise_and_widen(shape, dtype, group, zero_points, scale_dtype):
    g = torch.Generator("cuda").manual_seed(sum(shape) + group)
    w = (torch.randn(shape, generator=g, device="cuda") * torch.exp(torch.randn(*shape[:-1], 1, generator=g, device="cuda")))
    w[..., :8] *= 3
    w = w.to(dtype)
    w.view(-1, shape[-1])[0, :32] = 0
    if zero_points:
        w.view(-1, shape[-1])[-1] = w.view(-1, shape[-1])[-1].abs()
    q = m.int4_quantise(w, group=group, zero_points=zero_points, scale_dtype=scale_dtype)
    st = scale_dtype or (torch.bfloat16 if dtype == torch.float32 else dtype)
    codes, scales, zeros = quantised(w, group, zero_points, st)
    assert isinstance(q, m.Int4) and q.group == group
    assert torch.equal(q.scales, scales) and torch.equal(q.codes, codes)
    assert (q.zeros is None) if zeros is None else torch.equal(q.zeros, zeros)
    wide = m.int4_widen(q)
    assert wide.shape == w.shape and torch.equal(wide, values(q[:3], group).to(st))  # one rounding of an exact f32 product
    # each value within half a step of the scale (and the scale's rounding of the 15 steps; the ends may be cut by it)
    at = torch.arange(shape[-1], device="cuda") // group
    step = scales[..., at].double()
    assert ((values(q[:3], group) - w.double()).abs() <= step * (0.5 + 16 * torch.finfo(st).eps)).all()


def test_quantise_of_strided_rows_tiny_and_values_that_are_not_finite():
    g = torch.Generator("cuda").manual_seed(8)
    wide = torch.randn(20, 300, generator=g, device="cuda").bfloat16()[:, :296]
    with pytest.raises(m.MoeFFNError):  # rows 600 bytes apart
        m.int4_quantise(wide[:, 8:264], group=64)
    wide = torch.nn.functional.pad(wide, (0, 8))
    w = wide[:, 8:264]
    for zero_points in (False, True):
        q = m.int4_quantise(w, group=64, zero_points=zero_points)
        codes, scales, _ = quantised(w, 64, zero_points, torch.bfloat16)
        assert torch.equal(q.codes, codes) and torch.equal(q.scales, scales)
        bad = torch.randn(4, 128, generator=g, device="cuda")
        bad[0, 3], bad[1, 40], bad[2] = math.nan, -math.inf, 1e-30
        bad[3, 64:] = 3e38
        q = m.int4_quantise(bad, group=32, zero_points=zero_points, scale_dtype=torch.float16)
        assert torch.isinf(q.scales[0, 0]) and torch.isinf(q.scales[1, 1]) and torch.isinf(q.scales[3, 2:]).all()
        assert torch.isfinite(q.scales[0, 1:]).all() and torch.isfinite(q.scales[1, [0, 2, 3]]).all()
        assert (q.scales[2] == 2.0 ** -14).all() and (m.int4_widen(q)[2] == 0).all()
        x = torch.ones(1, 128, device="cuda", dtype=torch.float16)
        assert (~torch.isfinite(m.int4_matmul(x, q))).tolist() == [[True, True, False, True]]


def test_widened_weights_in_the_gated_block_and_codes_in_the_product():
    """A prompt takes the widened weights through gated_ffn, a token the codes: the same weights."""
    torch.manual_seed(4)
    hidden, inter = 256, 384
    ws = [m.int4_quantise(torch.randn(n, k, device="cuda") * k ** -0.5, group=64) for n, k in
          ((inter, hidden), (inter, hidden), (hidden, inter))]
    x = torch.randn(70, hidden, device="cuda").bfloat16()
    y = m.gated_ffn(x, *(m.int4_widen(w) for w in ws))
    g, u = m.int4_matmul(x, ws[0]), m.int4_matmul(x, ws[1])
    z = m.int4_matmul((torch.nn.functional.silu(g.float()) * u.float()).bfloat16(), ws[2])
    # 2-norm: the widened weights' roundings (of three matrices), g's, u's, h's and the results': each half a step of
    # 2^-8 at most, apart from one another
    assert (y.double() - z.double()).norm() <= math.sqrt(10) * 2.0 ** -8 * y.double().norm()


def test_refusals():
    x = torch.randn(4, 256, device="cuda").bfloat16()
    w = m.int4_quantise(torch.randn(64, 256, device="cuda"))
    half = m.int4_quantise(torch.randn(64, 256, device="cuda"), scale_dtype=torch.float16)
    for bad in (w._replace(codes=w.codes[:, :-1]), w._replace(scales=w.scales[:-1]), w._replace(scales=w.scales.float()),
                w._replace(zeros=torch.zeros(64, 3, device="cuda", dtype=torch.uint8)), w._replace(group=48), half,
                w._replace(codes=w.codes.view(torch.int8)), w._replace(codes=w.codes.cpu()),
                w._replace(codes=w.codes.T.contiguous().T), w._replace(codes=w.codes[0], scales=w.scales[0])):
        with pytest.raises(ValueError):
            m.int4_matmul(x, bad)
    for bad_x in (x.float(), x[:, :-32], x.T, x[0]):
        with pytest.raises(ValueError):
            m.int4_matmul(bad_x, w)
    with pytest.raises(TypeError):
        m.int4_matmul(x, None)
    with pytest.raises(TypeError):
        m.int4_matmul(x, (w.codes, None, None, 128))
    with pytest.raises(TypeError):
        m.int4_matmul(None, w, stream=torch.cuda.current_stream())
    with pytest.raises(ValueError):
        m.int4_matmul(x, torch.randn(64, 256, device="cuda").bfloat16())  # no codes
    with pytest.raises(m.MoeFFNError):
        m.int4_matmul(x[:0], w)
    with pytest.raises(m.MoeFFNError):  # rows that do not begin at 16 bytes
        m.int4_matmul(torch.randn(4, 300, device="cuda").bfloat16()[:, 1:257], w)
    with pytest.raises(m.MoeFFNError):
        m.int4_matmul(x, w, out=x[:, :64])
    for bad_w in (torch.randn(64, 250, device="cuda"), torch.randn(64, device="cuda"), torch.randn(64, 256),
                  torch.randn(64, 256, device="cuda").double(), torch.randn(2, 256, 64, device="cuda").transpose(1, 2)):
        with pytest.raises(ValueError):
            m.int4_quantise(bad_w)
    with pytest.raises(ValueError):
        m.int4_quantise(torch.randn(64, 256, device="cuda"), group=100)
    with pytest.raises(ValueError):
        m.int4_quantise(torch.randn(64, 256, device="cuda"), scale_dtype=torch.float32)
    with pytest.raises(ValueError):
        m.int4_widen(w, out=torch.empty(64, 256, device="cuda"))
