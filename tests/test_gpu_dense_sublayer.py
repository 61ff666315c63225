"""The dense sublayer's operators run together, as a layer of a model runs them: norm, gated block, residual
update fused with the next layer's norm; the same with FP8 projections; a training step through two layers;
and next to the routed block on one stream.

Tolerances: e = eps / 2 of bf16 bounds one rounding; a path's outputs differ from 64-bit arithmetic by the
roundings on the way (y, g and u or h, f, out), each at most e relative in 2-norm (a rounding's error is
independent of the value), through maps that here pass on relative errors with a factor of at most 2 (a norm
of a vector and a product of two factors): 12 e in 2-norm covers six of them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
E = 2.0 ** -8
HIDDEN, INTER = 512, 640


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def layer(gen):
    def n(*s, std=1.0):
        return torch.randn(*s, generator=gen, device="cuda") * std

    return dict(norm_in=1 + n(HIDDEN, std=0.1), norm_f=1 + n(HIDDEN, std=0.1), gate=(0.8 + n(HIDDEN, std=0.1)).to(BF16),
                w_gate=n(INTER, HIDDEN, std=HIDDEN ** -0.5).to(BF16), w_up=n(INTER, HIDDEN, std=HIDDEN ** -0.5).to(BF16),
                w_down=n(HIDDEN, INTER, std=INTER ** -0.5).to(BF16))


def rms(v, w):
    return v / (v.square().mean(1, keepdim=True) + 1e-6).sqrt() * w


def reference(state, layers):
    """The layers in 64 bits: rms norm, gated block, its output's norm times the gate onto the stream."""
    for w in layers:
        y = rms(state, w["norm_in"])
        g, u = y @ w["w_gate"].T, y @ w["w_up"].T
        state = state + 0.5 * w["gate"] * rms((g * torch.sigmoid(g) * u) @ w["w_down"].T, w["norm_f"])
    return state


def run(m, state, layers, save=False, ffn=None):
    kept = []
    out, y = m.block_norm(state, norm_next=layers[0]["norm_in"], block_dtype=BF16)
    for i, w in enumerate(layers):
        if ffn:
            f, saved = ffn(w, y), None
        elif save:
            f, saved = m.gated_ffn(y, w["w_gate"], w["w_up"], w["w_down"], save=True)
        else:
            f, saved = m.gated_ffn(y, w["w_gate"], w["w_up"], w["w_down"]), None
        after = layers[i + 1]["norm_in"] if i + 1 < len(layers) else None
        kept.append((out, y, f, saved))
        out, y = m.block_norm(out, f, norm_f=w["norm_f"], gate=w["gate"], residual_scale=0.5, norm_next=after)
        kept[-1] += (out, after)
    return out, kept


@pytest.mark.parametrize("rows", [1, 3, 7, 130, 1000])
def test_layers_forward(cuda_lib, rows):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(rows)
    layers = [layer(gen) for _ in range(3)]
    state = torch.randn(rows, HIDDEN, generator=gen, device="cuda")
    out, _ = run(m, state, layers)
    ref = reference(state.double(), [{k: v.double() for k, v in w.items()} for w in layers])
    assert rel(out - state, ref - state.double()) <= 12 * E
    assert m.dense_status() == 0


@pytest.mark.parametrize("rows", [2, 200])
def test_layers_in_fp8(cuda_lib, rows):
    # the reference takes the same FP8 weights; the activations' codes are off by 2^-4 relative at most,
    # two of them in series and about independent: 2 * 2^-4 in 2-norm, beside the bf16 roundings
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(rows)
    w = layer(gen)
    q = {k: m.fp8_quantise(w[k], block_rows=128) for k in ("w_gate", "w_up", "w_down")}
    wide = {k: (c.double() * s.double().repeat_interleave(128, 0)[:c.shape[0]].repeat_interleave(128, 1)[:, :c.shape[1]])
            for k, (c, s) in q.items()}

    def ffn(_, y):
        a, sa = m.fp8_quantise(y)
        g, u = (m.fp8_matmul(a, sa, *q[k], out_dtype=torch.float32) for k in ("w_gate", "w_up"))
        h, sh = m.fp8_quantise((g * torch.sigmoid(g) * u).to(BF16))
        return m.fp8_matmul(h, sh, *q["w_down"])

    state = torch.randn(rows, HIDDEN, generator=gen, device="cuda")
    out, _ = run(m, state, [w], ffn=ffn)
    ref = reference(state.double(), [{**{k: v.double() for k, v in w.items()}, **wide}])
    assert rel(out - state, ref - state.double()) <= 2 * 2.0 ** -4 + 12 * E


def test_training_step_through_two_layers(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(5)
    layers = [layer(gen) for _ in range(2)]
    state = torch.randn(300, HIDDEN, generator=gen, device="cuda")
    d_out = torch.randn(300, HIDDEN, generator=gen, device="cuda")

    def step():
        out, kept = run(m, state, layers, save=True)
        grads, d, d_y = [], d_out, None
        for w, (before, y, f, saved, after, norm_next) in zip(layers[::-1], kept[::-1]):
            b = m.block_norm_backward(after, f, norm_f=w["norm_f"], gate=w["gate"], residual_scale=0.5,
                                      norm_next=norm_next, d_out=d, d_y=d_y)
            g = m.gated_ffn_backward(y, w["w_gate"], w["w_up"], w["w_down"], saved, b["d_f"])
            d, d_y = b["d_state"], g["d_x"]
            grads.append({**b, **g})
        first = m.block_norm_backward(kept[0][0], norm_next=layers[0]["norm_in"], d_out=d, d_y=d_y)
        return out, grads[::-1], first

    out, grads, first = step()
    leaves = [{k: v.double().requires_grad_(True) for k, v in w.items()} for w in layers]
    s = state.double().requires_grad_(True)
    ref = reference(s, leaves)
    names = ("norm_f", "gate", "w_gate", "w_up", "w_down", "norm_in")
    got = torch.autograd.grad(ref, [s] + [w[k] for w in leaves for k in names], d_out.double())
    # twice the forward's roundings and as many backward
    assert rel(first["d_state"], got[0]) <= 24 * E
    for i, (w, g) in enumerate(zip(leaves, grads)):
        mine = {"norm_f": g["d_norm_f"], "gate": g["d_gate"], "w_gate": g["d_w_gate"], "w_up": g["d_w_up"],
                "w_down": g["d_w_down"], "norm_in": (first if i == 0 else grads[i - 1])["d_norm_next"]}
        for j, k in enumerate(names):
            assert rel(mine[k], got[1 + i * len(names) + j]) <= 24 * E, (i, k)
    # the whole step captured, beside the live tensors of the eager one, and replayed on other inputs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_out, g_grads, g_first = step()
    state.copy_(torch.randn(300, HIDDEN, generator=gen, device="cuda"))
    graph.replay()
    e_out, e_grads, e_first = step()
    torch.cuda.synchronize()
    assert torch.equal(g_out, e_out) and torch.equal(g_first["d_state"], e_first["d_state"])
    for a, b in zip(g_grads, e_grads):
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_two_streams_and_two_graphs_at_once(cuda_lib):
    # calls in flight together have workspaces of their own
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(6)
    layers = [layer(gen) for _ in range(2)]
    states = [torch.randn(r, HIDDEN, generator=gen, device="cuda") for r in (400, 2)]
    want = [run(m, s, layers)[0].clone() for s in states]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in states]
    for s in states:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(run(m, s, layers)[0])
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    eager = []
    for s, st in zip(states, streams):
        with torch.cuda.stream(st):
            eager.append(run(m, s, layers)[0])
    torch.cuda.synchronize()
    for w, o, e in zip(want, outs, eager):
        assert torch.equal(w, o) and torch.equal(w, e)


def test_beside_the_routed_block(cuda_lib):
    # a dense layer before a routed one on one stream: the routed block's results are what they were
    import synth
    from deepseek_v4_moe_gb300 import MoeFFN, config_from
    import deepseek_v4_moe_gb300 as m
    from synth.device import upload
    gen = torch.Generator(device="cuda").manual_seed(7)
    cfg = synth.CONFIGS["c0_tiny"]
    dev = upload(synth.Case(cfg), "cuda:0")
    h = MoeFFN(config_from(cfg), {cfg.layer: dev["weights"]})
    alone = h.forward(dev["state"], dev["token_ids"], cfg.layer).clone()
    layers = [layer(gen)]
    state = torch.randn(40, HIDDEN, generator=gen, device="cuda")
    first, _ = run(m, state, layers)
    between = h.forward(dev["state"], dev["token_ids"], cfg.layer)
    again, _ = run(m, state, layers)
    torch.cuda.synchronize()
    assert torch.equal(alone, between) and torch.equal(first, again) and h.status() == 0
    h.close()
