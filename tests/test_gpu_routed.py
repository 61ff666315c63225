"""The routed layer without a handle against 64-bit arithmetic."""
import math

import pytest
import torch

import deepseek_v4_moe_gb300 as m
from test_gpu_int4 import SUM_SLACK, make, values

pytestmark = pytest.mark.gpu


def plain(w):
    return values(w[:3], w.group) if isinstance(w, m.Int4) else w.double()


def act64(g, act):
    z = g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    return g * torch.sigmoid(z)


def routing(x, router, bias, top_k, score, normalise, scale):
    """Indices and weights in 64 bits, and the least gap between the values that decide about each token."""
    l = x.double() @ router.double().T
    s = torch.sigmoid(l) if score == "sigmoid" else l.softmax(1)
    rank = l if bias is None else s + bias.double()
    v, order = torch.sort(rank, dim=1, descending=True, stable=True)
    gaps = (v[:, :-1] - v[:, 1:])[:, :top_k]
    index = order[:, :top_k]
    w = s.gather(1, index)
    if normalise:
        w = w / w.sum(1, keepdim=True)
    return index, scale * w, gaps.amin(1) if gaps.shape[1] else torch.full_like(v[:, 0], math.inf)


def check(got, x, router, ws, top_k, shared, act, bias=None, score="sigmoid", normalise=True, scale=1.0):
    y, index, weight = got
    want_index, want_weight, gap = routing(x, router, bias, top_k, score, normalise, scale)
    # a logit in f32 is off by less than 2^-16 of its sum of magnitudes, whose mean is below 32 here
    sure = gap > 2.0 ** -11 * (1 if bias is None else 0.25)
    assert index.dtype == torch.int32 and weight.dtype == torch.float32
    assert sure.float().mean() > 0.5 and torch.equal(index[sure].long(), want_index[sure])
    index = index.long()
    s = x.double() @ router.double().T
    s = torch.sigmoid(s) if score == "sigmoid" else s.softmax(1)
    w = s.gather(1, index)
    w = scale * (w / w.sum(1, keepdim=True) if normalise else w)
    assert ((weight.double() - w).abs() <= 2.0 ** -11 * w).all()  # the logits' errors, as above
    xd, eps = x.double(), torch.finfo(x.dtype).eps / 2
    want, room = torch.zeros_like(xd), torch.zeros_like(xd)

    def add(e, mats, rows, weights):
        wg, wu, wd = (plain(v)[e] for v in mats) if not isinstance(mats[0], m.Int4) else (
            plain(m.Int4(v.codes[e], v.scales[e], v.zeros[e] if v.zeros is not None else None, v.group)) for v in mats)
        xr = xd[rows]
        g, u = xr @ wg.T, xr @ wu.T
        dg, du = (SUM_SLACK * (xr.abs() @ v.abs().T) for v in (wg, wu))
        a = act64(g, act)
        h = weights * a * u
        # act's slope is below 1.13; h is rounded to the type
        dh = weights.abs() * (1.13 * u.abs() * dg + (a.abs() + 1.13 * dg) * du) + (eps + 2.0 ** -16) * h.abs()
        if x.dtype == torch.float16:
            dh = dh + 2.0 ** -25
        want[rows] += h @ wd.T
        room[rows] += (dh + SUM_SLACK * h.abs()) @ wd.abs().T

    for e in index.unique().tolist():
        rows, slot = (index == e).nonzero(as_tuple=True)
        add(e, ws, rows, weight[rows, slot].double()[:, None])
    if shared:
        for e in range(shared[0].codes.shape[0] if isinstance(shared[0], m.Int4) else shared[0].shape[0]):
            add(e, shared, torch.arange(len(x), device="cuda"), torch.ones(len(x), 1, device="cuda", dtype=torch.float64))
    room = room + eps * want.abs()
    assert y.dtype == x.dtype and ((y.double() - want).abs() <= room * (1 + 2.0 ** -7) + 2.0 ** -25).all()
    # 2-norm: h's and y's roundings, half a step each at most and apart from one another
    assert (y.double() - want).norm() <= math.sqrt(2) * eps * want.norm()


CASES = [  # rows, hidden, inter, experts, top_k, shared, bits, group, zeros, dtype, score, bias, router in f32, act
    (1, 512, 256, 16, 2, 1, 16, 0, False, torch.bfloat16, "sigmoid", True, False, "silu"),
    (1, 64, 32, 1, 1, 0, 4, 32, True, torch.float16, "softmax", False, True, "silu"),
    (2, 1000, 424, 60, 4, 0, 16, 0, False, torch.float16, "softmax", False, False, "gelu"),
    (3, 1024, 96, 256, 6, 2, 4, 64, False, torch.bfloat16, "sigmoid", True, True, "silu"),
    (5, 72, 40, 33, 3, 1, 16, 0, False, torch.bfloat16, "softmax", True, True, "silu"),
    (7, 8, 8, 512, 8, 0, 16, 0, False, torch.float16, "sigmoid", False, False, "silu"),
    (8, 544, 288, 17, 5, 1, 4, 128, True, torch.float16, "sigmoid", False, False, "gelu"),
    (9, 256, 512, 8, 8, 8, 16, 0, False, torch.bfloat16, "softmax", False, False, "silu"),
    (12, 2080, 160, 64, 1, 0, 4, 32, False, torch.bfloat16, "softmax", True, False, "silu"),
    (16, 4096, 128, 300, 6, 1, 16, 0, False, torch.bfloat16, "sigmoid", True, False, "silu"),
    (17, 136, 2048, 4, 2, 1, 16, 0, False, torch.float16, "sigmoid", False, True, "gelu"),
    (25, 320, 96, 31, 7, 3, 4, 64, True, torch.bfloat16, "sigmoid", True, False, "silu"),
    (32, 264, 136, 128, 8, 1, 16, 0, False, torch.bfloat16, "softmax", False, False, "silu"),
    (32, 1056, 320, 5, 5, 0, 4, 128, False, torch.float16, "sigmoid", False, False, "silu")]


def layer(rows, hidden, inter, experts, shared, bits, group, zeros, dtype, router_f32, bias, seed=0):
    g = torch.Generator("cuda").manual_seed(seed + rows * 131 + hidden)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731

    def mats(count):
        if not count:
            return None
        shapes = ((count, inter, hidden), (count, inter, hidden), (count, hidden, inter))
        if bits == 4:
            return tuple(make(s, dtype, group, zeros, g) for s in shapes)
        return tuple((r(*s) * s[-1] ** -0.5).to(dtype) for s in shapes)

    x = r(rows, hidden).to(dtype)
    router = (r(experts, hidden) * 1.5 * hidden ** -0.5).to(torch.float32 if router_f32 else dtype)
    return x, router, mats(experts), mats(shared), 0.3 * r(experts) if bias else None


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}x{c[1]}x{c[2]}e{c[3]}k{c[4]}s{c[5]}b{c[6]}" for c in CASES])
def test_routed_ffn(case):
    rows, hidden, inter, experts, top_k, shared, bits, group, zeros, dtype, score, with_bias, router_f32, act = case
    x, router, ws, sh, bias = layer(rows, hidden, inter, experts, shared, bits, group, zeros, dtype, router_f32, with_bias)
    for normalise, scale in ((True, 1.0), (False, 2.5)):
        got = m.routed_ffn(x, router, *ws, top_k, bias=bias, score=score, normalise=normalise, route_scale=scale, shared=sh,
                           activation=act)
        check(got, x, router, ws, top_k, sh, act, bias, score, normalise, scale)


def test_ties_go_to_the_lower_index_and_masked_experts_come_last():
    x, router, ws, _, _ = layer(6, 64, 32, 40, 0, 16, 0, False, torch.bfloat16, False, False)
    router[1::2] = router[0::2]  # pairs of equal experts
    for score in ("sigmoid", "softmax"):
        for bias in (None, torch.zeros(40, device="cuda")):
            _, index, weight = m.routed_ffn(x, router, *ws, 6, bias=bias, score=score)
            assert (index[:, 0::2] + 1 == index[:, 1::2]).all() and (index[:, 0::2] % 2 == 0).all()
            assert torch.equal(weight[:, 0::2], weight[:, 1::2])
    _, index, _ = m.routed_ffn(x, torch.zeros_like(router), *ws, 8)
    assert torch.equal(index, torch.arange(8, device="cuda", dtype=torch.int32).expand(6, 8))
    _, index, _ = m.routed_ffn(-x.abs(), torch.zeros_like(router), *ws, 8)  # negative zeros
    assert torch.equal(index, torch.arange(8, device="cuda", dtype=torch.int32).expand(6, 8))
    bias = torch.full((40,), -math.inf, device="cuda")
    bias[[3, 17, 39]] = 0
    for score in ("sigmoid", "softmax"):
        y, index, weight = m.routed_ffn(x, router, *ws, 5, bias=bias, score=score)
        assert (index[:, :3].sort(1).values == torch.tensor([3, 17, 39], device="cuda")).all()
        assert torch.equal(index[:, 3:], torch.tensor([0, 1], device="cuda", dtype=torch.int32).expand(6, 2))
        assert torch.isfinite(y).all()


@pytest.mark.parametrize("size", [100.0, -100.0])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_logits_far_out(score, size):
    """Scores that are 1, or 0, in 32 bits: chosen by the logits, weighted by the scores' ratios."""
    x = torch.zeros(2, 64, device="cuda", dtype=torch.float16)
    x[:, 0] = 16
    router = torch.zeros(12, 64, device="cuda", dtype=torch.float32)
    router[:, 0] = (size + torch.arange(12, device="cuda") * 0.25) / 16
    ws = [torch.randn(s, device="cuda").half() * 0.1 for s in ((12, 32, 64), (12, 32, 64), (12, 64, 32))]
    y, index, weight = m.routed_ffn(x, router, *ws, 4, score=score)
    want_index, want, _ = routing(x, router, None, 4, score, True, 1.0)
    assert index.tolist() == [[11, 10, 9, 8]] * 2 == want_index.tolist()
    # a logit of 100 in f32 is off by 2^-17 at most, an exponential as much
    assert ((weight.double() - want).abs() <= 2.0 ** -15 * want).all() and torch.isfinite(y).all()


def test_a_token_that_is_not_finite_leaves_the_others():
    x, router, ws, sh, bias = layer(9, 128, 64, 12, 1, 16, 0, False, torch.bfloat16, False, True)
    y, index, weight = m.routed_ffn(x, router, *ws, 3, bias=bias, shared=sh)
    for value in (math.nan, math.inf):
        bad = x.clone()
        bad[4, 7] = value
        z, i, w = m.routed_ffn(bad, router, *ws, 3, bias=bias, shared=sh)
        keep = [t for t in range(9) if t != 4]
        assert torch.equal(z[keep], y[keep]) and torch.equal(i[keep], index[keep]) and torch.equal(w[keep], weight[keep])
        assert ((i[4] >= 0) & (i[4] < 12)).all() and len(set(i[4].tolist())) == 3 and not torch.isfinite(z[4]).all()


def test_strides_given_output_one_shared_expert_without_its_dimension():
    x, router, ws, sh, bias = layer(6, 256, 64, 10, 1, 16, 0, False, torch.bfloat16, False, False)
    want = m.routed_ffn(x, router, *ws, 3, shared=sh)
    wide = torch.zeros(6, 300, device="cuda", dtype=torch.bfloat16)[:, :296]
    with pytest.raises(m.MoeFFNError):  # rows 600 bytes apart
        m.routed_ffn(wide[:, 8:264], router, *ws, 3, shared=sh)
    wide = torch.zeros(6, 304, device="cuda", dtype=torch.bfloat16)
    wide[:, 8:264] = x
    out = torch.full((6, 301), 5.0, device="cuda", dtype=torch.bfloat16)
    got = m.routed_ffn(wide[:, 8:264], router, *ws, 3, shared=tuple(w[0] for w in sh), out=out[:, 1:257])
    assert got[0].data_ptr() == out[:, 1:257].data_ptr()
    assert torch.equal(out[:, 1:257], want[0]) and (out[:, 0] == 5).all() and (out[:, 257:] == 5).all()
    assert torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


def test_the_same_bits_on_two_streams_at_once_and_replayed():
    x, router, ws, sh, bias = layer(11, 1024, 512, 32, 1, 16, 0, False, torch.bfloat16, False, True)
    first = m.routed_ffn(x, router, *ws, 4, bias=bias, shared=sh)
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, kept = [], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            m.routed_ffn(x, router, *ws, 4, bias=bias, shared=sh)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                for _ in range(3):
                    out = m.routed_ffn(x, router, *ws, 4, bias=bias, shared=sh)
            graphs.append(graph)
            kept.append(out)
    torch.cuda.synchronize()
    for _ in range(5):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for out in kept:
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_offsets_past_32_bits():
    """Experts whose matrices lie past 2^32 bytes, reached by a bias."""
    experts, hidden, inter = 258, 4096, 2048
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(2, hidden, generator=g, device="cuda").bfloat16()
    router = torch.zeros(experts, hidden, device="cuda", dtype=torch.bfloat16)
    bias = torch.zeros(experts, device="cuda")
    bias[[256, 257]] = 1
    ws = []
    for s in ((experts, inter, hidden), (experts, inter, hidden), (experts, hidden, inter)):
        w = torch.zeros(s, device="cuda", dtype=torch.bfloat16)
        assert w[256:].data_ptr() - w.data_ptr() >= 2 ** 32
        w[256:] = torch.randn(2, *s[1:], generator=g, device="cuda") * s[-1] ** -0.5
        ws.append(w)
    y, index, weight = m.routed_ffn(x, router, *ws, 2, bias=bias)
    near = m.routed_ffn(x, router[256:].contiguous(), *(w[256:].clone() for w in ws), 2, bias=bias[256:].contiguous())
    assert index.tolist() == [[256, 257]] * 2 and torch.equal(y, near[0]) and y.float().norm() > 1


def test_decoder_layers_in_few_bits():
    """A run of layers as they are served: norm, the routed layer with 4-bit experts, norm, an FP8 gated block, norm in
    8 bits; captured and replayed, against the same layers in 64 bits on the operators' own operands."""
    torch.manual_seed(7)
    rows, hidden, inter, experts = 4, 512, 256, 16
    stream0 = torch.randn(rows, hidden, device="cuda")
    w1, w2 = (1 + 0.1 * torch.randn(hidden, device="cuda") for _ in range(2))
    router = torch.randn(experts, hidden, device="cuda") * 2 * hidden ** -0.5
    q = [m.int4_quantise(torch.randn(s, device="cuda") * s[-1] ** -0.5, group=64, zero_points=True) for s in
         ((experts, inter, hidden), (experts, inter, hidden), (experts, hidden, inter))]
    head = m.int4_quantise(torch.randn(1000, hidden, device="cuda") * hidden ** -0.5)
    gu8 = m.fp8_quantise(torch.randn(2 * inter, hidden, device="cuda") * hidden ** -0.5, block_rows=128)
    d8 = m.fp8_quantise(torch.randn(hidden, inter, device="cuda") * inter ** -0.5, block_rows=128)

    def step(state):
        _, y = m.block_norm(state, norm_next=w1, block_dtype=torch.bfloat16)
        f, index, weight = m.routed_ffn(y, router, *q, 4)
        out, codes, scales = m.block_norm_fp8(state, f, norm_next=w2)
        gu = m.fp8_matmul(codes, scales, *gu8)
        f2 = m.fp8_matmul(*m.gated_quantise(gu[:, :inter], gu[:, inter:]), *d8)
        final, y2 = m.block_norm(out, f2, norm_next=w1)
        return out, final, index, m.int4_matmul(y2, head), y, f, f2, y2

    state = stream0.clone()
    step(state)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            kept = step(state)
    torch.cuda.synchronize()
    state.copy_(torch.randn(rows, hidden, device="cuda"))
    graph.replay()
    torch.cuda.synchronize()
    eager = step(state)
    assert all(torch.equal(a, b) for a, b in zip(kept, eager))
    out, final, index, logits, y, f, f2, y2 = eager
    check((f, index, m.routed_ffn(y, router, *q, 4)[2]), y, router, q, 4, None, "silu")
    v = values(head[:3], head.group)
    assert ((logits.double() - y2.double() @ v.T).abs() <= 2.0 ** -8 * (y2.double() @ v.T).abs() * 1.01
            + SUM_SLACK * (y2.double().abs() @ v.abs().T)).all()
    # the stream: sums of what the blocks gave, in f32
    assert torch.equal(out, state + f.float()) and torch.equal(final, out + f2.float())


def test_refusals():
    x, router, ws, sh, bias = layer(4, 128, 64, 12, 1, 16, 0, False, torch.bfloat16, False, True)
    ok = dict(bias=bias, shared=sh)
    m.routed_ffn(x, router, *ws, 3, **ok)
    for args, kw in [((x.float(), router, *ws, 3), {}), ((x, router.half(), *ws, 3), {}), ((x, router[:11], *ws, 3), {}),
                     ((x, router, ws[0], ws[1][:, :32], ws[2], 3), {}), ((x, router, ws[0], ws[1], ws[0], 3), {}),
                     ((x, router, *ws, 3), dict(bias=bias[:5])), ((x, router, *ws, 3), dict(bias=bias.half())),
                     ((x, router, *ws, 3), dict(score="relu")), ((x, router, *ws, 3), dict(activation="relu")),
                     ((x, router, *ws, 3), dict(shared=sh[:2])), ((x, router, ws[0].half(), *ws[1:], 3), {}),
                     ((x, router, m.int4_quantise(ws[0]), *ws[1:], 3), {}),
                     ((x, router, *(m.int4_quantise(w, group=g) for w, g in zip(ws, (32, 64, 32))), 3), {}),
                     ((x, router, *ws, 3), dict(out=torch.empty(4, 127, device="cuda", dtype=torch.bfloat16)))]:
        with pytest.raises(ValueError):
            m.routed_ffn(*args, **{**ok, **kw})
    many = torch.randn(33, 128, device="cuda").bfloat16()
    for args, kw in [((many, router, *ws, 3), {}), ((x[:0], router, *ws, 3), {}), ((x, router, *ws, 0), {}),
                     ((x, router, *ws, 9), {}), ((x, router, *ws, 3), dict(out=x))]:
        with pytest.raises(m.MoeFFNError):
            m.routed_ffn(*args, **{**ok, **kw})
    few = layer(2, 64, 32, 3, 0, 16, 0, False, torch.bfloat16, False, False)
    with pytest.raises(m.MoeFFNError):
        m.routed_ffn(few[0], few[1], *few[2], 4)  # more choices than experts
    with pytest.raises(TypeError):
        m.routed_ffn(x, router, None, *ws[1:], 3)
