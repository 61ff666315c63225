"""The dense feed-forward sublayer's operators, for measurement: the norms around a block with its gate and
residual scale (block_norm), the gated feed-forward block (gated_ffn) and the FP8 product with block scales
(fp8_matmul, with fp8_quantise, which makes its operands), each forward and, where a model trains through it,
backward.

``own`` selects between the plain form (elementary torch operations in 32 bits) and the framework's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
EPS = 1e-6
BLOCK = 128
GELU_C = math.sqrt(2.0 / math.pi)


def _cdiv(a, b):
    return -(-a // b)


def listed():
    return [
        # one token of a decode step: the block's output joins the f32 stream and the next norm is taken
        dict(name="norm_token", op="norm", dir="fwd", rows=1, hidden=4096, stream="f32", block="bf16", gate="none",
             post=True, next=True),
        # a padded batch of a small model, all in bf16, a gate value for each token; hidden is no power of two
        dict(name="norm_ragged", op="norm", dir="fwd", rows=1777, hidden=1000, stream="bf16", block="bf16",
             gate="token", post=True, next=True),
        # a training step's backward with a learned gate vector that every row shares
        dict(name="norm_train", op="norm", dir="bwd", rows=4096, hidden=4096, stream="f32", block="bf16",
             gate="vector", post=True, next=True),
        # one token of a decode step through the block
        dict(name="ffn_token", op="ffn", dir="fwd", rows=1, hidden=4096, inter=2048, type="bf16", act="silu"),
        # a 4096-token prompt
        dict(name="ffn_prompt", op="ffn", dir="fwd", rows=4096, hidden=4096, inter=2048, type="bf16", act="silu"),
        # a short ragged batch of a small fp16 model in training: no size a whole number of tiles
        dict(name="ffn_ragged", op="ffn", dir="bwd", rows=333, hidden=1000, inter=1416, type="f16", act="gelu"),
        # a training step's backward at the prompt's size
        dict(name="ffn_train", op="ffn", dir="bwd", rows=4096, hidden=4096, inter=2048, type="bf16", act="silu"),
        # one token through one projection
        dict(name="fp8_token", op="fp8", rows=1, n=4096, k=4096, a="e4m3", b="e4m3", out="bf16"),
        # a prompt through one projection
        dict(name="fp8_prompt", op="fp8", rows=4096, n=4096, k=4096, a="e4m3", b="e4m3", out="bf16"),
        # a ragged batch into an odd number of outputs (a head); K ends inside a block
        dict(name="fp8_ragged", op="fp8", rows=77, n=1031, k=2000, a="e4m3", b="e4m3", out="f32"),
        # a prompt's activations made into operands: a scale for each token and 128 values
        dict(name="quantise_prompt", op="quantise", rows=4096, k=4096, type="bf16", tall=1, pow2=False, code="e4m3"),
        # a weight matrix made into an operand: a scale for each 128 x 128 values, ragged at both ends
        dict(name="quantise_weight", op="quantise", rows=2000, k=4112, type="f32", tall=128, pow2=True, code="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "ffn", "ffn", "ffn", "fp8", "fp8", "quantise"])
    if op == "norm":
        block = rng.choice(["bf16", "bf16", "f16", "f32"])
        hidden = _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            hidden = _cdiv(hidden, 8) * 8
        gate = rng.choice(["none", "vector", "token", "full", "group"])
        rows = _log_int(rng, 1, 4096)
        if gate == "group":  # a gate vector for each sequence of a batch
            rows = _cdiv(rows, 4) * 4
        post, nxt = rng.choice([(True, True), (True, False), (False, True)])
        return dict(op="norm", dir=rng.choice(["fwd", "bwd"]), rows=rows, hidden=hidden,
                    stream=rng.choice(["f32", block]), block=block, gate=gate, post=post, next=nxt)
    if op == "ffn":
        return dict(op="ffn", dir=rng.choice(["fwd", "fwd", "bwd"]), rows=_log_int(rng, 1, 4096),
                    hidden=8 * _log_int(rng, 16, 512), inter=8 * _log_int(rng, 16, 256),
                    type=rng.choice(["bf16", "bf16", "f16"]), act=rng.choice(["silu", "silu", "gelu"]))
    if op == "fp8":
        return dict(op="fp8", rows=_log_int(rng, 1, 4096), n=_log_int(rng, 128, 8192), k=16 * _log_int(rng, 8, 512),
                    a=rng.choice(["e4m3", "e4m3", "e5m2"]), b=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    out=rng.choice(["bf16", "bf16", "f16", "f32"]))
    return dict(op="quantise", rows=_log_int(rng, 1, 4096), k=16 * _log_int(rng, 8, 512),
                type=rng.choice(["bf16", "f16", "f32"]), tall=rng.choice([1, 128]), pow2=rng.choice([False, True]),
                code=rng.choice(["e4m3", "e4m3", "e5m2"]))


# ---- inputs ----------------------------------------------------------------------------------------------


def _codes(x, code, tall):
    """An operand as a program keeps it: codes and a scale for each block of `tall` x 128 values."""
    rows, k = x.shape
    rb, kb = _cdiv(rows, tall), _cdiv(k, BLOCK)
    full = torch.zeros(rb * tall, kb * BLOCK, device=x.device)
    full[:rows, :k] = x
    tiles = full.view(rb, tall, kb, BLOCK)
    scale = (tiles.abs().amax(dim=(1, 3)) / FP8_MAX[code]).clamp_min(1e-30)
    q = (tiles / scale[:, None, :, None]).reshape(rb * tall, kb * BLOCK)[:rows, :k]
    return q.contiguous().to(FP8[code]), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    c, st = case, {"case": dict(case)}
    if c["op"] == "norm":
        rows, hidden, ts, tb = c["rows"], c["hidden"], DTYPES[c["stream"]], DTYPES[c["block"]]
        # a stream has a few channels far larger than the rest
        spread = torch.exp(normal(hidden, std=0.5))
        st["state"] = (normal(rows, hidden) * spread).to(ts)
        st["f"] = (normal(rows, hidden) * torch.exp(normal(rows, 1, std=0.3))).to(tb)
        st["w_post"] = 1 + normal(hidden, std=0.1) if c["post"] else None
        st["w_next"] = 1 + normal(hidden, std=0.1) if c["next"] else None
        shape = {"none": None, "vector": (hidden,), "token": (rows, 1), "full": (rows, hidden),
                 "group": (4, hidden)}[c["gate"]]
        st["gate"] = (0.5 + normal(*shape, std=0.2)).to(tb) if shape else None
        st["scale"] = 0.7
        if c["dir"] == "bwd":
            st["d_out"] = normal(rows, hidden).to(ts)
            st["d_y"] = normal(rows, hidden).to(tb) if c["next"] else None
    elif c["op"] == "ffn":
        rows, hidden, inter, t = c["rows"], c["hidden"], c["inter"], DTYPES[c["type"]]
        x = normal(rows, hidden).to(t)
        wg, wu = (normal(inter, hidden, std=hidden ** -0.5).to(t) for _ in range(2))
        wd = normal(hidden, inter, std=inter ** -0.5).to(t)
        st.update(x=x, w_gate=wg, w_up=wu, w_down=wd)
        if c["dir"] == "bwd":  # what the forward pass kept
            st["gate"] = (x.float() @ wg.float().T).to(t)
            st["up"] = (x.float() @ wu.float().T).to(t)
            st["d_y"] = normal(rows, hidden).to(t)
    elif c["op"] == "fp8":
        rows, n, k = c["rows"], c["n"], c["k"]
        a = normal(rows, k) * torch.exp(normal(rows, 1, std=0.5)) * torch.exp(normal(k, std=0.5))
        st["a"], st["a_scale"] = _codes(a, c["a"], 1)
        st["b"], st["b_scale"] = _codes(normal(n, k, std=k ** -0.5), c["b"], BLOCK)
    else:
        x = normal(c["rows"], c["k"]) * torch.exp(normal(c["rows"], 1, std=0.5)) * torch.exp(normal(c["k"], std=0.5))
        st["x"] = x.to(DTYPES[c["type"]])
    return st


# ---- one pass --------------------------------------------------------------------------------------------


def run(st):
    return {"norm": _norm, "ffn": _ffn, "fp8": _fp8, "quantise": _quantise}[st["case"]["op"]](st)


def _gate_rows(gate, rows, hidden):
    """The gate as [rows or 1, hidden or 1], a row for each of the stream's rows."""
    if gate.dim() == 2 and gate.shape[0] not in (1, rows):
        return gate.repeat_interleave(rows // gate.shape[0], dim=0)
    return gate.view(1, hidden) if gate.dim() == 1 else gate


def _norm(st):
    c, f, gate, scale = st["case"], st["f"], st["gate"], st["scale"]
    w_post, w_next = st["w_post"], st["w_next"]
    if own:
        import deepseek_v4_moe_gb300 as m
        if c["dir"] == "fwd":
            return m.block_norm(st["state"], f, norm_f=w_post, gate=gate, residual_scale=scale, norm_next=w_next,
                                eps=EPS)
        d = m.block_norm_backward(st["state"], f, norm_f=w_post, gate=gate, residual_scale=scale, norm_next=w_next,
                                  eps=EPS, d_out=st["d_out"], d_y=st["d_y"])
        return d
    rows, hidden = f.shape
    f32 = f.float()
    rf = torch.rsqrt(f32.square().mean(1, keepdim=True) + EPS) if w_post is not None else 1.0
    n = f32 * rf * (w_post if w_post is not None else 1.0)
    gr = _gate_rows(gate.float(), rows, hidden) if gate is not None else 1.0
    if c["dir"] == "fwd":
        out = (st["state"].float() + scale * gr * n).to(st["state"].dtype)
        y = None
        if w_next is not None:
            s = out.float()
            y = (s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * w_next).to(f.dtype)
        return out, y
    # backward: st["state"] holds the stream after the block (what the forward pass wrote)
    d = {}
    ds = st["d_out"].float()
    if w_next is not None:
        s, gy = st["state"].float(), st["d_y"].float()
        rs = torch.rsqrt(s.square().mean(1, keepdim=True) + EPS)
        gw = gy * w_next
        ds = ds + rs * (gw - s * rs.square() * (gw * s).mean(1, keepdim=True))
        d["d_norm_next"] = (gy * s * rs).sum(0)
    d["d_state"] = ds.to(st["state"].dtype)
    dn = scale * gr * ds
    if gate is not None:
        dg = scale * n * ds
        if c["gate"] == "token":
            dg = dg.sum(1, keepdim=True)
        elif c["gate"] == "vector":
            dg = dg.sum(0)
        elif c["gate"] == "group":
            dg = dg.view(gate.shape[0], -1, hidden).sum(1)
        d["d_gate"] = dg.to(gate.dtype)
    if w_post is not None:
        d["d_norm_f"] = (dn * f32 * rf).sum(0)
        dw = dn * w_post
        dn = rf * (dw - f32 * rf.square() * (dw * f32).mean(1, keepdim=True))
    d["d_f"] = dn.to(f.dtype)
    return d


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    t = torch.tanh(GELU_C * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * g * g)


def _ffn(st):
    c = st["case"]
    x, wg, wu, wd = st["x"], st["w_gate"], st["w_up"], st["w_down"]
    if own:
        import deepseek_v4_moe_gb300 as m
        if c["dir"] == "fwd":
            return m.gated_ffn(x, wg, wu, wd, activation=c["act"])
        return m.gated_ffn_backward(x, wg, wu, wd, (st["gate"], st["up"]), st["d_y"], activation=c["act"])
    t = x.dtype
    x, wg, wu, wd = x.float(), wg.float(), wu.float(), wd.float()
    if c["dir"] == "fwd":
        return ((_act(x @ wg.T, c["act"])[0] * (x @ wu.T)) @ wd.T).to(t)
    u, dy = st["up"].float(), st["d_y"].float()
    a, da = _act(st["gate"].float(), c["act"])
    dh = dy @ wd
    dg, du = dh * u * da, dh * a
    return {"d_x": (dg @ wg + du @ wu).to(t), "d_w_gate": (dg.T @ x).to(t), "d_w_up": (du.T @ x).to(t),
            "d_w_down": (dy.T @ (a * u)).to(t)}


def _spread(scale, tall, rows, k):
    return scale.repeat_interleave(tall, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :k]


def _fp8(st):
    c = st["case"]
    if own:
        import deepseek_v4_moe_gb300 as m
        return m.fp8_matmul(st["a"], st["a_scale"], st["b"], st["b_scale"], out_dtype=DTYPES[c["out"]])
    a = st["a"].float() * _spread(st["a_scale"], 1, *st["a"].shape)
    b = st["b"].float() * _spread(st["b_scale"], BLOCK, *st["b"].shape)
    return (a @ b.T).to(DTYPES[c["out"]])


def _quantise(st):
    c, x = st["case"], st["x"]
    if own:
        import deepseek_v4_moe_gb300 as m
        return m.fp8_quantise(x, block_rows=c["tall"], pow2_scales=c["pow2"], dtype=FP8[c["code"]])
    (rows, k), tall, most = x.shape, c["tall"], FP8_MAX[c["code"]]
    rb, kb = _cdiv(rows, tall), _cdiv(k, BLOCK)
    full = torch.zeros(rb * tall, kb * BLOCK, device=x.device)
    full[:rows, :k] = x
    amax = full.view(rb, tall, kb, BLOCK).abs().amax(dim=(1, 3))
    scale = torch.where(amax == 0, torch.ones_like(amax), (amax / most).clamp_min(2.0 ** -126))
    if c["pow2"]:  # up to the next power of two
        m, e = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(scale), torch.where(m == 0.5, e - 1, e))
    q = (full[:rows, :k] / _spread(scale, tall, rows, k)).clamp(-most, most)
    return q.to(FP8[c["code"]]), scale


# ---- what a pass cannot do without -----------------------------------------------------------------------


def work(case):
    c = case
    if c["op"] == "norm":
        rows, hidden, s, b = c["rows"], c["hidden"], SIZE[c["stream"]], SIZE[c["block"]]
        gate = {"none": 0, "vector": hidden, "token": rows, "full": rows * hidden, "group": 4 * hidden}[c["gate"]] * b
        norms = 4 * hidden * (int(c["post"]) + int(c["next"]))
        one = rows * hidden
        if c["dir"] == "fwd":
            return {"bytes": one * (2 * s + b + b * int(c["next"])) + gate + norms, "flops": 10 * one}
        # reads d_out, f, and (for the next norm) the stream and d_y; writes d_state and d_f
        return {"bytes": one * (2 * s + 2 * b + (s + b) * int(c["next"])) + 2 * gate + 2 * norms, "flops": 25 * one}
    if c["op"] == "ffn":
        rows, hidden, inter = c["rows"], c["hidden"], c["inter"]
        w = 3 * hidden * inter
        if c["dir"] == "fwd":
            return {"bytes": 2 * (w + 2 * rows * hidden), "flops": 2 * rows * w}
        return {"bytes": 2 * (2 * w + 3 * rows * hidden + 2 * rows * inter), "flops": 4 * rows * w}
    if c["op"] == "fp8":
        rows, n, k = c["rows"], c["n"], c["k"]
        kb = _cdiv(k, BLOCK)
        return {"bytes": (rows + n) * k + 4 * kb * (rows + _cdiv(n, BLOCK)) + SIZE[c["out"]] * rows * n,
                "flops": 2 * rows * n * k}
    rows, k = c["rows"], c["k"]
    return {"bytes": rows * k * (SIZE[c["type"]] + 1) + 4 * _cdiv(rows, c["tall"]) * _cdiv(k, BLOCK),
            "flops": 4 * rows * k}


# ---- the definitions in 64 bits --------------------------------------------------------------------------


def _stored(v, dtype):
    """v (64 bits) as a tensor of `dtype` holds it, in 64 bits again."""
    return v.to(dtype).double()


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "norm":
        f = st["f"].double().requires_grad_(True)
        wp = st["w_post"].double().requires_grad_(True) if c["post"] else None
        wn = st["w_next"].double().requires_grad_(True) if c["next"] else None
        gate = st["gate"].double().requires_grad_(True) if st["gate"] is not None else None
        rows, hidden = f.shape

        def rms(v, w):
            return v / (v.pow(2).sum(1, keepdim=True) / hidden + EPS).sqrt() * w

        branch = rms(f, wp) if wp is not None else f
        if gate is not None:
            branch = branch * {"vector": lambda: gate.expand(rows, hidden), "token": lambda: gate,
                               "full": lambda: gate,
                               "group": lambda: gate[torch.arange(rows, device="cuda") // (rows // 4)]}[c["gate"]]()
        branch = branch * st["scale"]
        if c["dir"] == "fwd":
            out = (st["state"].double() + branch).detach()
            y = rms(_stored(out, st["state"].dtype), wn).detach() if wn is not None else None
            return out, y
        # the stream after the block is given; its gradient goes on to the stream before it and to the branch
        s = st["state"].double().requires_grad_(True)
        d = {}
        ds = st["d_out"].double()
        if wn is not None:
            gs, d["d_norm_next"] = torch.autograd.grad(rms(s, wn), (s, wn), st["d_y"].double())
            ds = ds + gs
        d["d_state"] = ds
        leaves = {"d_f": f, "d_gate": gate, "d_norm_f": wp}
        leaves = {k: v for k, v in leaves.items() if v is not None}
        d.update(zip(leaves, torch.autograd.grad(branch, list(leaves.values()), ds)))
        return d
    if c["op"] == "ffn":
        x, wg, wu, wd = (st[k].double() for k in ("x", "w_gate", "w_up", "w_down"))

        def act(g):
            if c["act"] == "silu":
                return g / (1 + (-g).exp())
            return g * 0.5 * (1 + ((2 / math.pi) ** 0.5 * (g + 0.044715 * g.pow(3))).tanh())

        if c["dir"] == "fwd":
            return (act(x @ wg.T) * (x @ wu.T)) @ wd.T
        g = st["gate"].double().requires_grad_(True)
        u = st["up"].double().requires_grad_(True)
        dy = st["d_y"].double()
        h = act(g) * u
        dg, du = torch.autograd.grad(h, (g, u), dy @ wd)
        return {"d_x": torch.cat([dg, du], 1) @ torch.cat([wg, wu], 0), "d_w_gate": dg.T @ x, "d_w_up": du.T @ x,
                "d_w_down": dy.T @ h.detach()}
    if c["op"] == "fp8":
        a, b = st["a"].double(), st["b"].double()
        sa, sb = st["a_scale"].double(), st["b_scale"].double()
        col = torch.arange(a.shape[1], device="cuda") // BLOCK
        row = torch.arange(b.shape[0], device="cuda") // BLOCK
        return (a * sa[:, col]) @ (b * sb[row][:, col]).T
    x, most = st["x"].double(), FP8_MAX[c["code"]]
    rows, k = x.shape
    pad = torch.nn.functional.pad(x, (0, -k % BLOCK, 0, -rows % c["tall"]))
    tiles = pad.unflatten(1, (-1, BLOCK)).unflatten(0, (-1, c["tall"]))
    amax = tiles.abs().flatten(3).amax(3).amax(1)
    scale = (amax / most).clamp_min(2.0 ** -126)
    if c["pow2"]:
        e = torch.floor(torch.log2(scale))
        e = torch.where(torch.exp2(e) < scale, e + 1, e)
        e = torch.where(torch.exp2(e - 1) >= scale, e - 1, e)
        scale = torch.exp2(e)
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    at = torch.arange(rows, device="cuda") // c["tall"]
    v = x / scale[at][:, torch.arange(k, device="cuda") // BLOCK]
    # the nearest value of the format, even mantissas at ties
    bits, low = {"e4m3": (3, -6), "e5m2": (2, -14)}[c["code"]]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - bits)
    return (torch.round(v / step) * step).clamp(-most, most), scale
