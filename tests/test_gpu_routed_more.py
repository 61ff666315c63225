"""The routed layer without a handle, further: the choice's place in shared memory, magnitudes at the types' ends, the
precision of the hidden values, weights that are not finite, and the choice of every token."""
import ctypes
import math

import pytest
import torch

import deepseek_v4_moe_gb300 as m
import test_gpu_int4 as t4
import test_gpu_routed as tr
from deepseek_v4_moe_gb300 import _lib

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


def fine_layer(rows, bits, dtype, down=1.0, inter=32):
    """Small sums, so that what the hidden values lose shows: one expert of each token."""
    x, router, ws, _, _ = tr.layer(rows, 64, inter, 8, 0, bits, 32, True, dtype, True, False, seed=3)
    if bits == 16:
        return x, router, [*ws[:2], ws[2] * down]
    return x, router, [*ws[:2], ws[2]._replace(scales=ws[2].scales * down)]


def fine_room(x, router, ws, index, weight, lost):
    """y in 64 bits, and the room that its parts leave: lost(h, the token's largest |h|) of the hidden values.  Sums of 64
    exact products in f32, four steps of 16 with a unit of 2^-23 each and as much again where planes and groups are joined:
    2^-20 of the sum of magnitudes."""
    want = torch.zeros(len(x), ws[2].scales.shape[1] if isinstance(ws[2], m.Int4) else ws[2].shape[1], device="cuda",
                       dtype=torch.float64)
    room, xd = torch.zeros_like(want), x.double()
    for e in index.unique().tolist():
        g, u, d = ((t4.values((w.codes[e], w.scales[e], w.zeros[e] if w.zeros is not None else None), w.group)
                    if isinstance(w, m.Int4) else w[e].double()) for w in ws)
        by = (weight.double() * (index == e)).sum(1, keepdim=True)
        a, b = xd @ g.T, xd @ u.T
        da, db = (2.0 ** -20 * (xd.abs() @ v.abs().T) for v in (g, u))
        s = torch.nn.functional.silu(a)
        h = by * s * b
        dh = by * (1.13 * b.abs() * da + (s.abs() + 1.13 * da) * db) + 2.0 ** -19 * h.abs()
        dh = dh + lost(h.abs() + dh, (h.abs() + dh).amax(1, keepdim=True))
        want += h @ d.T
        room += (dh + 2.0 ** -20 * h.abs()) @ d.abs().T
    return want, (room + torch.finfo(x.dtype).eps / 2 * want.abs()) * (1 + 2.0 ** -10)


# What the hidden values lose: as 16-bit numbers of two parts half a step of the second, 2^-18 of a value (f16: 2^-22, and
# of subnormal numbers 2^-25 2^-11); as three planes half a step of the third, 2^-12 of a value or 2^-27 of the largest.
LOST = {(16, BF16): lambda h, most: 2.0 ** -18 * h, (16, F16): lambda h, most: 2.0 ** -22 * h + 2.0 ** -36,
        (4, BF16): lambda h, most: torch.maximum(2.0 ** -12 * h, 2.0 ** -27 * most),
        (4, F16): lambda h, most: torch.maximum(2.0 ** -12 * h, 2.0 ** -27 * most)}


@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 23, 24, 25, 32])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("bits", [16, 4])
def test_hidden_values_keep_more_than_the_type(bits, dtype, rows):
    x, router, ws = fine_layer(rows, bits, dtype)
    y, index, weight = m.routed_ffn(x, router, *ws, 1)
    want, room = fine_room(x, router, ws, index, weight, LOST[bits, dtype])
    assert ((y.double() - want).abs() <= room + (2.0 ** -25 if dtype == F16 else 0)).all()


@pytest.mark.parametrize("bits", [16, 4])
def test_hidden_values_below_f16s_normal_numbers(bits):
    """Unnormalised weights of 0.004 take the hidden values to 10^-5, where a number of f16 has a few bits; large down
    matrices bring them back."""
    x, router, ws = fine_layer(20, bits, F16, down=64.0)
    x, router = x / 16, torch.cat([router[:8] * 0.01, torch.zeros(248, 64, device="cuda")])
    many = [torch.cat([w] * 32) if bits == 16 else w._replace(codes=torch.cat([w.codes] * 32), scales=torch.cat([w.scales] * 32),
                                                              zeros=torch.cat([w.zeros] * 32)) for w in ws]
    y, index, weight = m.routed_ffn(x, router, *many, 1, score="softmax", normalise=False)
    assert (weight < 0.005).all()
    want, room = fine_room(x, router, many, index, weight, LOST[bits, F16])
    assert want.abs().mean() > 2.0 ** -14  # (normal numbers again)
    assert ((y.double() - want).abs() <= room + 2.0 ** -25).all()


@pytest.mark.parametrize("bits", [16, 4])
def test_a_workspace_aligned_to_16_bytes(cuda_lib, bits):
    rows, hidden, inter, experts = 9, 256, 96, 10
    x, router, ws, _, _ = tr.layer(rows, hidden, inter, experts, 0, bits, 32, True, BF16, False, False)
    want = m.routed_ffn(x, router, *ws, 3)
    y, index = torch.empty_like(x), torch.empty(rows, 3, device="cuda", dtype=torch.int32)
    mats = [_lib.MoeFfnMatrices(*(t.data_ptr() for t in w[:3])) if bits == 4 else _lib.MoeFfnMatrices(w.data_ptr(), None, None)
            for w in ws]
    a = _lib.MoeFfnRoutedArgs(rows=rows, hidden=hidden, inter=inter, experts=experts, top_k=3, shared=0, type=_lib.TYPE_BF16,
                              router_type=_lib.TYPE_BF16, bits=bits, group=32, score=_lib.SCORES["sigmoid"], normalise=1,
                              activation=0, route_scale=1.0, x=x.data_ptr(), ld_x=hidden, router=router.data_ptr(),
                              gate=mats[0], up=mats[1], down=mats[2], y=y.data_ptr(), ld_y=hidden, indices=index.data_ptr())
    need = cuda_lib.moe_ffn_routed_workspace(ctypes.byref(a))
    space = torch.empty(need + 272, device="cuda", dtype=torch.uint8)
    a.workspace, a.workspace_bytes = (space.data_ptr() + 255) // 256 * 256 + 16, need
    stream = torch.cuda.current_stream().cuda_stream
    assert cuda_lib.moe_ffn_routed_forward(ctypes.byref(a), stream) == 0, cuda_lib.moe_ffn_last_error(None)
    assert torch.equal(y, want[0]) and torch.equal(index, want[1])


def spoil(w, e, row, column, value):
    """A value of expert e's matrix, or in 4 bits the scale of its group."""
    if isinstance(w, m.Int4):
        w.scales[e, row, column // w.group] = value
    else:
        w[e, row, column] = value


@pytest.mark.parametrize("rows,hidden,inter,shared", [(20, 256, 160, 1), (5, 4096, 64, 0), (32, 544, 96, 2), (2, 32, 32, 1)])
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_weights_that_are_not_finite_reach_the_tokens_that_chose_them(rows, hidden, inter, shared, bits, dtype):
    """Infinities and NaN in one expert: tokens of the others are as without them, up to the order of their sums."""
    x, router, ws, sh, _ = tr.layer(rows, hidden, inter, 6, shared, bits, 32, True, dtype, False, False)
    clean = m.routed_ffn(x, router, *ws, 2, shared=sh)
    bad = clean[1][0, 0].item()
    has = (clean[1] == bad).any(1)
    others = [w._replace(scales=w.scales.clone()) if bits == 4 else w.clone() for w in ws]
    spoil(others[2], bad, 3, 5, math.inf)
    spoil(others[2], bad, hidden - 1, inter - 1, math.nan)
    y, index, weight = m.routed_ffn(x, router, *others, 2, shared=sh)
    assert torch.equal(index, clean[1]) and torch.equal(weight, clean[2])
    assert not torch.isfinite(y[has][:, [3, hidden - 1]]).any() and has.any()
    rest = [c for c in range(hidden) if c not in (3, hidden - 1)]
    assert torch.equal(y[:, rest], clean[0][:, rest])
    if (~has).any():
        tr.check((y[~has], index[~has], weight[~has]), x[~has], router, ws, 2, sh, "silu")
    # a row of gate or up: all of y, of the expert's tokens alone
    spoil(others[1], bad, 7, 9, -math.inf)
    y, _, _ = m.routed_ffn(x, router, *others, 2, shared=sh)
    assert not torch.isfinite(y[has]).any()
    if (~has).any():
        tr.check((y[~has], index[~has], weight[~has]), x[~has], router, ws, 2, sh, "silu")


def test_weights_that_are_not_finite_in_a_shared_expert_reach_all():
    for bits in (16, 4):
        x, router, ws, sh, _ = tr.layer(9, 256, 96, 6, 1, bits, 64, False, BF16, False, False)
        clean = m.routed_ffn(x, router, *ws, 2, shared=sh)[0]
        spoil(sh[2], 0, 100, 50, math.nan)
        y = m.routed_ffn(x, router, *ws, 2, shared=sh)[0]
        rest = [c for c in range(256) if c != 100]
        assert torch.isnan(y[:, 100]).all() and torch.equal(y[:, rest], clean[:, rest])


@pytest.mark.parametrize("rows,hidden,experts,top_k", [(1, 4096, 256, 6), (32, 4096, 256, 8), (32, 1024, 512, 8), (31, 96, 33, 7),
                                                       (17, 32, 8, 8), (9, 65536, 5, 2), (26, 512, 64, 1)])
@pytest.mark.parametrize("score,with_bias,router_f32", [("sigmoid", True, False), ("sigmoid", False, True), ("softmax", True, True),
                                                        ("softmax", False, False)])
@pytest.mark.parametrize("bits", [16, 4])
def test_the_choice_of_every_token(bits, score, with_bias, router_f32, rows, hidden, experts, top_k):
    """Also of tokens whose experts lie so close that 32 bits may order them otherwise: no chosen expert is worse than one left
    out, and no slot than the next, by more than the logits' errors."""
    x, router, ws, _, bias = tr.layer(rows, hidden, 32, experts, 0, bits, 32, False, BF16, router_f32, with_bias, seed=11)
    _, index, weight = m.routed_ffn(x, router, *ws, top_k, bias=bias, score=score)
    i = index.long()
    assert ((i >= 0) & (i < experts)).all()
    assert all(len(set(row)) == top_k for row in i.tolist())
    l = x.double() @ router.double().T
    # a lane's sums of hidden / 256 values, then 13 levels: of 65536 values below 2^-15.9 of the magnitudes
    off = 2.0 ** -15.9 * (x.double().abs() @ router.double().abs().T).amax(1, keepdim=True)
    s = torch.sigmoid(l) if score == "sigmoid" else l.softmax(1)
    rank = l
    if with_bias:  # scores move by less than logits do, and by three roundings of their own
        rank, off = s + bias.double(), off + 2.0 ** -20
    got = rank.gather(1, i)
    left_out = rank.scatter(1, i, -math.inf).amax(1, keepdim=True)
    assert (got >= left_out - 2 * off).all()
    assert (got[:, :-1] >= got[:, 1:] - 2 * off).all()
    w = s.gather(1, i)
    w = w / w.sum(1, keepdim=True)
    off = 2.0 ** -15.9 * (x.double().abs() @ router.double().abs().T).amax(1, keepdim=True)
    assert ((weight.double() - w).abs() <= (4 * off + 2.0 ** -20) * w).all()  # a ratio of exponentials of two logits
    alone = torch.cat([m.routed_ffn(x[t:t + 1], router, *ws, top_k, bias=bias, score=score)[1] for t in range(rows)])
    assert torch.equal(alone, index)  # a token's choice does not depend on the others


# a bf16 layer of up to eight tokens in groups of 32: tiles of eight groups, two at a time; hidden and inter that end inside
# a tile of 256 columns, and more units than SMs
SHORT = [(1, 4128, 160, 40, 6, 1, 32, False, BF16, "sigmoid", True, False, "silu"),
         (5, 1056, 1312, 24, 4, 0, 32, True, BF16, "softmax", False, True, "gelu"),
         (8, 288, 2080, 30, 8, 2, 32, True, BF16, "sigmoid", False, False, "silu"),
         (8, 32, 64, 8, 2, 1, 32, False, BF16, "sigmoid", True, False, "silu")]


@pytest.mark.parametrize("case", SHORT, ids=[f"{c[0]}x{c[1]}x{c[2]}" for c in SHORT])
def test_few_tokens_in_short_groups(case, cuda_lib):
    rows, hidden, inter, experts, top_k, shared, group, zeros, dtype, score, bias, router_f32, act = case
    x, router, ws, sh, b = tr.layer(rows, hidden, inter, experts, shared, 4, group, zeros, dtype, router_f32, bias, seed=7)

    def call():
        return m.routed_ffn(x, router, *ws, top_k, bias=b, score=score, shared=sh, activation=act)

    want = call()
    tr.check(want, x, router, ws, top_k, sh, act, b, score)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(call())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = call()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for g in [*got, kept] for a, c in zip(g, want))
    assert cuda_lib.moe_ffn_dense_fault_injection(1, 20000) == 0
    try:
        call()
        assert m.dense_status() == 8
    finally:
        cuda_lib.moe_ffn_dense_fault_injection(0, 0)
    assert all(torch.equal(a, c) for a, c in zip(call(), want)) and m.dense_status() == 0
