"""Products with 4-bit weights in their FP8 form, and the routed layer, where they can go wrong: sizes on either side of each
choice of a kernel, magnitudes far apart, rows that are not finite, shares of k without a tile, zeros, calls on two streams
at once, captured ones, and waits that run out."""
import ctypes

import pytest
import torch

import deepseek_v4_moe_gb300 as m
import test_gpu_int4 as t4
import test_gpu_routed as tr
from deepseek_v4_moe_gb300 import _lib

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def splits_x(lib, rows, n, k, group, dtype):
    a = _lib.MoeFfnInt4MatmulArgs(rows=rows, n=n, k=k, type=_lib.TYPE_F16 if dtype == F16 else _lib.TYPE_BF16, group=group)
    return lib.moe_ffn_int4_matmul_workspace(ctypes.byref(a)) > 0


def product(rows, n, k, group, zeros, dtype, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + rows * 7919 + n * 31 + k)
    return torch.randn(rows, k, generator=g, device="cuda").to(dtype), t4.make((n, k), dtype, group, zeros, g)


# A row's planes lose at most 2^-22 of its largest magnitude for each value: with normal values, whose largest is below 6
# times their mean magnitude, below 2^-19 of the sum of magnitudes, which the other tests' room for sums (2^-16) holds.
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("rows,n,k,group", [(1, 8193, 4096, 128), (8, 16500, 2048, 128), (9, 33000, 1024, 128), (16, 130, 8192, 64),
                                            (12, 40, 16352, 128), (16, 8200, 8224, 64), (1, 10000, 6752, 64), (17, 1, 32, 32),
                                            (33, 2049, 352, 128), (18, 5000, 416, 32), (100, 333, 1184, 64)])
def test_int4_matmul_on_planes(cuda_lib, rows, n, k, group, zeros, dtype):
    assert splits_x(cuda_lib, rows, n, k, group, dtype)
    x, w = product(rows, n, k, group, zeros, dtype)
    t4.check_product(m.int4_matmul(x, w), x, w)


FORMS = [(3, 300, 512, 128), (20, 300, 512, 128), (16, 130, 8192, 64)]  # on mma.sync, and on planes of 32 and of 16 tokens


@pytest.mark.parametrize("rows,n,k,group", FORMS)
@pytest.mark.parametrize("power", [-100, -40, 60, 110])
def test_powers_of_two_pass_through(rows, n, k, group, power):
    """Rows times a power of two: every step is exact up to it, so the results' bits are the same but for the exponent."""
    x, w = product(rows, n, k, group, True, BF16)
    x = torch.where(x.abs() < 2.0 ** -8, 2.0 ** -8, x)  # (bf16: no value leaves the normal numbers at 2^-100)
    y = m.int4_matmul(x, w)
    assert torch.equal(m.int4_matmul(x * 2.0 ** power, w), (y.double() * 2.0 ** power).to(BF16))
    each = torch.tensor([2.0 ** (power * (i % 2)) for i in range(rows)], device="cuda")[:, None]
    assert torch.equal(m.int4_matmul((x * each).to(BF16), w), (y.double() * each).to(BF16))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("rows,n,k,group", FORMS)
def test_one_large_value_beside_small_ones(rows, n, k, group, dtype):
    """A value 2^12 times the others, in a column whose weights are 0: what is lost of the others is at most half a step of
    the last plane, 2^-22 of the largest magnitude (f16: 2^-27), for each."""
    x, w = product(rows, n, k, group, False, dtype)
    w.codes[:, 3] = w.codes[:, 3] & 0x0F | 0x80  # column 7: code 8, which is 0
    big = 2.0 ** 12
    x[:, 7] = big
    y = m.int4_matmul(x, w)
    v = t4.values(w[:3], w.group)
    x = x.double()
    want = x @ v.T
    x[:, 7] = 0
    room = torch.finfo(dtype).eps / 2 * want.abs() + t4.SUM_SLACK * (x.abs() @ v.abs().T) + (2.0 ** -25 if dtype == F16 else 0)
    # the group of column 7: its zero point is taken off sums that hold the large value, in f32 units of at most
    # 2^-23 of 2^12 times 8, some tens of times
    lost = (2.0 ** -22 if dtype == BF16 else 2.0 ** -27) * big * v.abs().sum(1)
    lost = lost + 64 * 2.0 ** -23 * 8 * big * w.scales[:, 0].double()
    assert ((y.double() - want).abs() <= (room + lost) * (1 + 2.0 ** -7)).all()


@pytest.mark.parametrize("rows,n,k,group", FORMS[1:])
def test_rows_that_are_not_finite_are_nan_and_leave_the_others(rows, n, k, group):
    x, w = product(rows, n, k, group, True, F16)
    y = m.int4_matmul(x, w)
    bad = x.clone()
    bad[1, 5], bad[4, k - 1], bad[9, 0] = float("inf"), float("nan"), -float("inf")
    z = m.int4_matmul(bad, w)
    some = [1, 4, 9]
    rest = [i for i in range(rows) if i not in some]
    assert z[some].isnan().all() and torch.equal(z[rest], y[rest])
    x[2] = 0
    assert (m.int4_matmul(x, w)[2] == 0).all()


# few-bit layers: shares of the down product without a tile, one tile of everything, every tokens' width and group
LAYERS = [(1, 4096, 32, 1, 1, 0, 128, False, BF16, "sigmoid", False, False, "silu"),
          (1, 32, 32, 3, 2, 1, 32, True, F16, "softmax", True, True, "gelu"),
          (8, 1024, 2048, 16, 2, 1, 64, False, F16, "sigmoid", False, False, "silu"),
          (7, 8224, 96, 9, 3, 1, 64, True, BF16, "sigmoid", True, True, "silu"),
          (16, 2048, 544, 40, 8, 2, 128, True, BF16, "sigmoid", True, False, "silu"),
          (11, 160, 992, 12, 4, 8, 32, True, F16, "softmax", False, False, "gelu"),
          (17, 512, 1056, 20, 3, 0, 32, True, F16, "sigmoid", False, True, "silu"),
          (32, 4128, 96, 256, 8, 1, 128, False, BF16, "softmax", True, False, "silu"),
          (32, 288, 2080, 6, 6, 8, 64, True, BF16, "sigmoid", False, False, "gelu"),
          (3, 20000, 64, 4, 2, 1, 32, False, F16, "sigmoid", False, False, "silu")]


@pytest.mark.parametrize("case", LAYERS, ids=[f"{c[0]}x{c[1]}x{c[2]}e{c[3]}k{c[4]}s{c[5]}g{c[6]}" for c in LAYERS])
@pytest.mark.parametrize("bits", [4, 16])
def test_routed_layers(case, bits):
    rows, hidden, inter, experts, top_k, shared, group, zeros, dtype, score, bias, router_f32, act = case
    x, router, ws, sh, b = tr.layer(rows, hidden, inter, experts, shared, bits, group, zeros, dtype, router_f32, bias, seed=5)
    got = m.routed_ffn(x, router, *ws, top_k, bias=b, score=score, route_scale=1.5, shared=sh, activation=act)
    tr.check(got, x, router, ws, top_k, sh, act, b, score, True, 1.5)


@pytest.mark.parametrize("bits", [4, 16])
def test_tokens_that_are_zero_or_not_finite(bits):
    x, router, ws, sh, _ = tr.layer(20, 256, 160, 24, 1, bits, 64, True, BF16, False, False)
    y, index, weight = m.routed_ffn(x, router, *ws, 3, shared=sh)
    z = x.clone()
    z[3], z[7, 100], z[19, 0] = 0, float("nan"), float("inf")
    y2, index2, weight2 = m.routed_ffn(z, router, *ws, 3, shared=sh)
    rest = [i for i in range(20) if i not in (3, 7, 19)]
    assert torch.equal(y2[rest], y[rest]) and torch.equal(index2[rest], index[rest]) and torch.equal(weight2[rest], weight[rest])
    assert (y2[3] == 0).all() and not y2[7].isfinite().any() and not y2[19].isfinite().any()


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_an_expert_whose_hidden_values_are_small_beside_anothers(dtype):
    """Two experts of each token, the one's hidden values 2^-12 of the other's and its down matrix 2^10 larger: a token's
    planes have one power of two, so of its hidden values up to 2^-22 (f16: 2^-27) of the largest is lost."""
    x, router, ws, _, _ = tr.layer(12, 256, 320, 2, 0, 4, 64, False, dtype, False, False)
    gate, up, down = ws
    up.scales[1] *= 2.0 ** -7
    gate.scales[1] *= 2.0 ** -2
    down.scales[1] *= 2.0 ** 4
    y, index, weight = m.routed_ffn(x, router, *ws, 2)
    want = torch.zeros_like(y, dtype=torch.float64)
    room = torch.zeros_like(want)
    eps = torch.finfo(dtype).eps / 2
    most = torch.zeros(len(x), 1, device="cuda", dtype=torch.float64)
    lose = torch.zeros_like(want)
    for e in range(2):
        g, u, d = (t4.values((t.codes[e], t.scales[e], None), t.group) for t in ws)
        a, b = x.double() @ g.T, x.double() @ u.T
        w = (weight.double() * (index == e)).sum(1, keepdim=True)
        h = torch.nn.functional.silu(a) * b * w
        da, db = (t4.SUM_SLACK * (x.double().abs() @ t.abs().T) for t in (g, u))
        dh = w.abs() * (1.13 * b.abs() * da + (a.abs() + 1.13 * da) * db) + (eps + 2.0 ** -16) * h.abs()
        dh = dh + (2.0 ** -25 if dtype == F16 else 0)
        want += h @ d.T
        room += (dh + t4.SUM_SLACK * h.abs()) @ d.abs().T
        most = torch.maximum(most, (h.abs() + dh).amax(1, keepdim=True))
        lose += d.abs().sum(1)
    room = room + eps * want.abs() + (2.0 ** -22 if dtype == BF16 else 2.0 ** -27) * most * lose
    assert ((y.double() - want).abs() <= room * (1 + 2.0 ** -7) + 2.0 ** -25).all()


def calls():
    """Every kernel of these operators: name, and a call that gives its results."""
    out = []
    for name, args in (("products", (3, 300, 512, 64, True, BF16)), ("planes", (20, 300, 4096, 128, False, F16)),
                       ("planes16", (16, 130, 8192, 64, True, BF16)), ("long", (60, 20000, 512, 128, False, BF16))):
        x, w = product(*args)
        out.append((name, lambda x=x, w=w: [m.int4_matmul(x, w)]))
    for bits, rows in ((16, 5), (16, 20), (4, 5), (4, 13), (4, 30)):
        x, router, ws, sh, b = tr.layer(rows, 512, 320, 24, 1, bits, 64, False, BF16, False, True)
        out.append((f"layer{bits}x{rows}", lambda a=(x, router, *ws), b=b, sh=sh: list(m.routed_ffn(*a, 3, bias=b, shared=sh))))
    return out


def test_two_streams_at_once_and_replayed():
    for name, call in calls():
        want = call()
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in range(2)]
        got = []
        for _ in range(4):
            for s in streams:
                with torch.cuda.stream(s):
                    got.append(call())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept = [call(), call()]
        for _ in range(3):
            for k in kept:
                for t in k:
                    t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            got += [[t.clone() for t in k] for k in kept]
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want)), name


def test_waits_that_run_out(cuda_lib):
    """CTA 0 of each kernel gives up after 20 ms; the next call finds everything in order."""
    for name, call in calls():
        good = call()
        assert m.dense_status() == 0
        assert cuda_lib.moe_ffn_dense_fault_injection(1, 20000) == 0
        try:
            call()
            assert m.dense_status() == 8, name
        finally:
            cuda_lib.moe_ffn_dense_fault_injection(0, 0)
        again = call()
        assert m.dense_status() == 0 and all(torch.equal(a, b) for a, b in zip(again, good)), name


def test_a_workspace_that_is_too_small_is_refused(cuda_lib):
    x, w = product(20, 64, 256, 128, False, BF16)
    out = torch.empty(20, 64, device="cuda", dtype=BF16)
    a = _lib.MoeFfnInt4MatmulArgs(rows=20, n=64, k=256, type=_lib.TYPE_BF16, group=128, x=x.data_ptr(), ld_x=256,
                                  codes=w.codes.data_ptr(), scales=w.scales.data_ptr(), out=out.data_ptr(), ld_out=64)
    need = cuda_lib.moe_ffn_int4_matmul_workspace(ctypes.byref(a))
    ws = torch.empty(need, device="cuda", dtype=torch.uint8)
    assert cuda_lib.moe_ffn_int4_matmul(ctypes.byref(a), None) == _lib.ERR_NULL_PTR
    a.workspace, a.workspace_bytes = ws.data_ptr(), need - 1
    assert cuda_lib.moe_ffn_int4_matmul(ctypes.byref(a), None) == _lib.ERR_NO_MEMORY
    a.workspace_bytes = need
    stream = torch.cuda.current_stream().cuda_stream
    assert cuda_lib.moe_ffn_int4_matmul(ctypes.byref(a), stream) == 0
    assert torch.equal(out, m.int4_matmul(x, w))
