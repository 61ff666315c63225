"""block_norm_fp8 and gated_quantise against 64-bit arithmetic.

A code has to be the nearest value of its format to y / scale, but for y's own error in 32 bits: the format's half step,
and a small relative error ``slack`` of the quotient.
"""
import math

import pytest
import torch

import deepseek_v4_moe_gb300 as m

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0, 3, -6), "e5m2": (torch.float8_e5m2, 57344.0, 2, -14)}
# A sum of squares (at most 16 terms a thread, 9 levels of a tree), rsqrt and three products: below 2^5 units of 2^-24.
NORM_SLACK = 2.0 ** -19


def _blocks(v):
    return torch.nn.functional.pad(v, (0, -v.shape[1] % 128)).unflatten(1, (-1, 128))


def check_codes(codes, scales, y, code, pow2, slack):
    """codes and scales of y (64 bits, relative error `slack`, a number or a tensor of y's shape)."""
    dtype, most, bits, low = FP8[code]
    rows, k = y.shape
    assert codes.dtype == dtype and codes.shape == y.shape and scales.shape == (rows, -(-k // 128))
    slack = torch.as_tensor(slack, device=y.device, dtype=torch.float64).expand(y.shape)
    amax, s = _blocks(y.abs()).amax(2), scales.double()
    want = torch.where(amax == 0, torch.ones_like(amax), (amax / most).clamp_min(2.0 ** -126))
    off = _blocks(slack).amax(2) + 2.0 ** -23
    if pow2:
        assert torch.equal(torch.exp2(torch.log2(s).round()), s)
        assert (s >= want * (1 - off)).all() and (s < 2 * want * (1 + off)).all()
    else:
        assert ((s - want).abs() <= off * want).all()
    v = y / s.repeat_interleave(128, 1)[:, :k]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - bits)
    # the quotient's own rounding, and a value whose error takes it over a power of two, where the step doubles
    room = step * (0.5 + 2.0 ** -10) + 2 * slack * v.abs()
    assert ((codes.double() - v).abs() <= room).all()


def _rms(v, w, eps):
    return v * torch.rsqrt(v.square().mean(1, keepdim=True) + eps) * w


SIZES = [(1, 1), (3, 7), (17, 64), (2, 100), (33, 127), (5, 128), (9, 129), (300, 512), (7, 1000), (6, 1001), (40, 1032),
         (2, 4095), (161, 4096), (3, 4104), (2, 8191), (5, 8192)]


@pytest.mark.parametrize("rows,hidden", SIZES)
@pytest.mark.parametrize("stream,block,gate,post,code,pow2", [
    (torch.float32, torch.bfloat16, "none", True, "e4m3", False),
    (torch.bfloat16, torch.bfloat16, "vector", True, "e5m2", True),
    (torch.float16, torch.float16, "token", False, "e4m3", True),
    (torch.float32, torch.float32, "group", True, "e4m3", False)])
def test_block_norm_fp8(rows, hidden, stream, block, gate, post, code, pow2):
    g = torch.Generator("cuda").manual_seed(rows * 10007 + hidden)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    state, f = r(rows, hidden).to(stream), (2 * r(rows, hidden)).to(block)
    wp, wn = 1 + 0.1 * r(hidden) if post else None, 1 + 0.1 * r(hidden)
    shape = {"none": None, "vector": (hidden,), "token": (rows, 1), "group": (rows, hidden)}[gate]
    gv = (0.5 + 0.2 * r(*shape)).to(block) if shape else None
    out, codes, scales = m.block_norm_fp8(state, f, norm_f=wp, gate=gv, residual_scale=0.7, norm_next=wn, eps=1e-5,
                                          pow2_scales=pow2, dtype=FP8[code][0])
    n = f.double()
    if post:
        n = _rms(n, wp.double(), 1e-5)
    branch = 0.7 * n * (gv.double() if gv is not None else 1.0)
    want = state.double() + branch
    # out: one rounding to its type, and the branch's error in 32 bits
    assert out.dtype == stream
    room = torch.finfo(stream).eps / 2 * want.abs() + NORM_SLACK * branch.abs() + 2.0 ** -24 * state.double().abs()
    if stream == torch.float16:
        room = room + 2.0 ** -25  # half a step of its subnormal values
    assert ((out.double() - want).abs() <= room * (1 + 2.0 ** -8)).all()
    check_codes(codes, scales, _rms(out.double(), wn.double(), 1e-5), code, pow2, NORM_SLACK)


def test_block_norm_fp8_without_block_in_place_and_strided():
    g = torch.Generator("cuda").manual_seed(3)
    wide = torch.randn(37, 1500, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(1000, generator=g, device="cuda")
    for first in (0, 8, 3):  # the last without wide accesses
        state = wide[:, first:first + 1000]
        got, codes, scales = m.block_norm_fp8(state, norm_next=w)
        assert got is state or got.data_ptr() == state.data_ptr()
        check_codes(codes, scales, _rms(state.double(), w.double(), 1e-6), "e4m3", False, NORM_SLACK)
    f = torch.randn(37, 1000, generator=g, device="cuda").bfloat16()
    state = wide[:, :1000].clone()
    apart = m.block_norm_fp8(state, f, norm_next=w)
    into = wide.clone()
    here = m.block_norm_fp8(into[:, :1000], f, norm_next=w, out=into[:, :1000])
    assert torch.equal(into[:, :1000], apart[0]) and torch.equal(into[:, 1000:], wide[:, 1000:])
    # rows 6000 bytes apart are no multiples of 32: read without wide accesses, the row is summed in another order than
    # the contiguous one, so the scales need not be the same bits
    for _, codes, scales in (here, apart):
        check_codes(codes, scales, _rms(apart[0].double(), w.double(), 1e-6), "e4m3", False, NORM_SLACK)


@pytest.mark.parametrize("hidden", [256, 1000, 257])
def test_block_norm_fp8_zeros_and_values_that_are_not_finite(hidden):
    state = torch.randn(4, hidden, device="cuda")
    state[0] = 0
    state[2, 3] = math.nan
    state[3, 5] = math.inf
    w = torch.ones(hidden, device="cuda")
    _, codes, scales = m.block_norm_fp8(state, norm_next=w)
    assert (codes[0].float() == 0).all() and (scales[0] == 1).all()
    check_codes(codes[1:2], scales[1:2], _rms(state[1:2].double(), w.double(), 1e-6), "e4m3", False, NORM_SLACK)
    assert torch.isnan(scales[2]).all()  # a norm of NaN
    assert torch.isnan(scales[3, 0]) and (scales[3, 1:] == 1).all()  # inf * 0; the rest divided by an infinite norm


@pytest.mark.parametrize("rows,inter", [(1, 1), (3, 100), (17, 128), (2, 1000), (333, 1416), (5, 1001), (64, 2048),
                                        (1, 8192), (7, 40000), (2000, 130)])
@pytest.mark.parametrize("dtype,act,code,pow2", [(torch.bfloat16, "silu", "e4m3", False), (torch.float16, "gelu", "e5m2", True),
                                                 (torch.float16, "silu", "e4m3", True)])
def test_gated_quantise(rows, inter, dtype, act, code, pow2):
    g = torch.Generator("cuda").manual_seed(rows * 31 + inter)
    gu = (2 * torch.randn(rows, 2 * inter, generator=g, device="cuda")).to(dtype)
    gate, up = gu[:, :inter], gu[:, inter:]
    codes, scales = m.gated_quantise(gate, up, activation=act, pow2_scales=pow2, dtype=FP8[code][0])
    a = gate.double()
    z = a if act == "silu" else 2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)
    # the sigmoid: a few units of 2^-22, and |z| 2^-23 of the exponent's rounding (twice as much for gelu's polynomial)
    check_codes(codes, scales, a * torch.sigmoid(z) * up.double(), code, pow2, (8 + 2 * z.abs()) * 2.0 ** -22)


def test_gated_quantise_zeros_and_values_that_are_not_finite():
    g = torch.ones(3, 300, device="cuda", dtype=torch.bfloat16)
    u = torch.ones_like(g)
    u[0] = 0
    u[1, 140] = math.nan
    g[2, 290] = math.inf
    codes, scales = m.gated_quantise(g, u)
    assert (codes[0].float() == 0).all() and (scales[0] == 1).all()
    assert torch.isfinite(scales[1, [0, 2]]).all() and torch.isnan(scales[1, 1])
    assert torch.isfinite(scales[2, :2]).all() and torch.isinf(scales[2, 2])
    assert (codes[2, 256:290].float() == 0).all()  # over an infinite scale


def test_fp8_gated_block_captured_on_another_stream():
    """Norm, product, gated product, product, as one layer in FP8 runs: captured and replayed on new inputs."""
    torch.manual_seed(5)
    rows, hidden, inter = 19, 512, 384
    state, f = torch.randn(rows, hidden, device="cuda"), torch.randn(rows, hidden, device="cuda").bfloat16()
    w = torch.ones(hidden, device="cuda")
    wgu = torch.randn(2 * inter, hidden, device="cuda") * hidden ** -0.5
    wd = torch.randn(hidden, inter, device="cuda") * inter ** -0.5
    qgu, sgu = m.fp8_quantise(wgu, block_rows=128)
    qd, sd = m.fp8_quantise(wd, block_rows=128)

    def layer():
        out, c, s = m.block_norm_fp8(state, f, norm_next=w)
        gu = m.fp8_matmul(c, s, qgu, sgu)
        c, s = m.gated_quantise(gu[:, :inter], gu[:, inter:])
        return out, m.fp8_matmul(c, s, qd, sd)

    layer()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = layer()
    torch.cuda.current_stream().wait_stream(side)
    f.copy_(torch.randn(rows, hidden, device="cuda"))
    graph.replay()
    out, y = layer()
    assert torch.equal(kept[0], out) and torch.equal(kept[1], y)
    # against 64 bits: each operand in e4m3 is off by 2^-5 of its value at most, 2^-5 / sqrt(3) on average
    x = _rms(out.double(), w.double(), 1e-6)
    gu = x @ wgu.double().T
    want = (torch.nn.functional.silu(gu[:, :inter]) * gu[:, inter:]) @ wd.double().T
    # 2-norm: two operands of each of two products and the product's growth through the gate: below 4 * 2^-5
    assert (y.double() - want).norm() <= 4 * 2.0 ** -5 * want.norm()


def test_refusals():
    x = torch.randn(4, 256, device="cuda")
    w = torch.ones(256, device="cuda")
    with pytest.raises(ValueError):
        m.block_norm_fp8(x, norm_next=w, dtype=torch.float16)
    with pytest.raises(ValueError):
        m.block_norm_fp8(x, norm_next=w[:255])
    with pytest.raises(ValueError):
        m.block_norm_fp8(x, gate=w, norm_next=w)
    with pytest.raises(ValueError):
        m.gated_quantise(x, x)
    h = x.half()
    with pytest.raises(ValueError):
        m.gated_quantise(h, h[:, :255])
    with pytest.raises(ValueError):
        m.gated_quantise(h, h.bfloat16())
    with pytest.raises(ValueError):
        m.gated_quantise(h, h, activation="relu")
    with pytest.raises(ValueError):
        m.gated_quantise(h.T, h.T)
    with pytest.raises(m.MoeFFNError):
        m.gated_quantise(h[:0], h[:0])
    with pytest.raises(TypeError):
        m.gated_quantise(None, h, stream=torch.cuda.current_stream())
