"""Serving a feed-forward sublayer in few bits and for a few tokens, for measurement: the norms around a block with
their output in FP8 (block_norm_fp8), the gated product in FP8 (gated_quantise), products with 4-bit weights and group
scales (int4_matmul), making and widening such weights (int4_quantise, int4_widen), and a whole mixture-of-experts
layer for a few tokens (routed_ffn).

``own`` selects between the plain form (elementary torch operations in 32 bits) and the framework's kernels.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
LEAST = {"bf16": 2.0 ** -126, "f16": 2.0 ** -14}  # the smallest normal value: no scale of a group is below it
EPS = 1e-6
BLOCK = 128
GELU_C = math.sqrt(2.0 / math.pi)


def _cdiv(a, b):
    return -(-a // b)


def listed():
    return [
        # one token of a decode step between two FP8 products: the block's output joins the f32 stream
        dict(name="norm8_token", op="norm", rows=1, hidden=4096, stream="f32", block="bf16", gate="none", post=True,
             pow2=False, code="e4m3"),
        # a 4096-token prompt there
        dict(name="norm8_prompt", op="norm", rows=4096, hidden=4096, stream="f32", block="bf16", gate="none",
             post=True, pow2=False, code="e4m3"),
        # a small ragged batch of a small fp16 model: the width ends inside a block
        dict(name="gated8_ragged", op="gated", rows=333, inter=1416, type="f16", act="gelu", pow2=True, code="e4m3"),
        # a 4096-token prompt between the products of an FP8 gated block
        dict(name="gated8_prompt", op="gated", rows=4096, inter=2048, type="bf16", act="silu", pow2=False,
             code="e4m3"),
        # one token through one projection
        dict(name="int4_token", op="int4", rows=1, n=4096, k=4096, type="bf16", group=128, zeros=False),
        # a decode batch into an odd number of outputs, with zero points and short groups
        dict(name="int4_ragged", op="int4", rows=13, n=1031, k=2016, type="f16", group=32, zeros=True),
        # a decode batch through the head over the whole vocabulary
        dict(name="int4_head", op="int4", rows=16, n=129280, k=4096, type="bf16", group=128, zeros=False),
        # a projection's weights made into codes, and widened again for a prompt
        dict(name="weights4_matrix", op="weights4", n=4096, k=2048, type="bf16", group=128, zeros=False),
        # the same with zero points, of sizes that are no multiples of a tile
        dict(name="weights4_ragged", op="weights4", n=1031, k=2016, type="f16", group=32, zeros=True),
        # one token of a decode step through a layer of 256 experts and a shared one
        dict(name="routed_token", op="routed", rows=1, hidden=4096, inter=2048, experts=256, top_k=6, shared=1,
             type="bf16", bits=16, group=128, zeros=False, score="sigmoid", bias=True, act="silu"),
        # a decode batch through the same layer with 4-bit weights
        dict(name="routed_batch4", op="routed", rows=16, hidden=4096, inter=2048, experts=256, top_k=6, shared=1,
             type="bf16", bits=4, group=128, zeros=False, score="sigmoid", bias=True, act="silu"),
        # a few tokens through a small layer whose sizes are no multiples of a tile
        dict(name="routed_ragged", op="routed", rows=5, hidden=1000, inter=424, experts=60, top_k=4, shared=0,
             type="f16", bits=16, group=128, zeros=False, score="softmax", bias=False, act="gelu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "gated", "int4", "int4", "weights4", "routed", "routed", "routed"])
    if op == "norm":
        block = rng.choice(["bf16", "bf16", "f16", "f32"])
        hidden, rows = _log_int(rng, 64, 8192), _log_int(rng, 1, 4096)
        if rng.random() < 0.7:
            hidden = _cdiv(hidden, 16) * 16
        return dict(op="norm", rows=rows, hidden=hidden, stream=rng.choice(["f32", block]), block=block,
                    gate=rng.choice(["none", "vector", "token"]), post=rng.random() < 0.7, pow2=rng.random() < 0.3,
                    code=rng.choice(["e4m3", "e4m3", "e5m2"]))
    if op == "gated":
        inter = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:
            inter = _cdiv(inter, 16) * 16
        return dict(op="gated", rows=_log_int(rng, 1, 4096), inter=inter, type=rng.choice(["bf16", "bf16", "f16"]),
                    act=rng.choice(["silu", "silu", "gelu"]), pow2=rng.random() < 0.3,
                    code=rng.choice(["e4m3", "e4m3", "e5m2"]))
    if op == "int4":
        return dict(op="int4", rows=_log_int(rng, 1, 64), n=_log_int(rng, 128, 16384), k=32 * _log_int(rng, 4, 256),
                    type=rng.choice(["bf16", "bf16", "f16"]), group=rng.choice([32, 64, 128, 128]),
                    zeros=rng.random() < 0.4)
    if op == "weights4":
        return dict(op="weights4", n=_log_int(rng, 128, 8192), k=32 * _log_int(rng, 4, 256),
                    type=rng.choice(["bf16", "bf16", "f16"]), group=rng.choice([32, 64, 128, 128]),
                    zeros=rng.random() < 0.4)
    bits = rng.choice([4, 16])
    step = 32 if bits == 4 else 8
    experts = _log_int(rng, 4, 256)
    return dict(op="routed", rows=_log_int(rng, 1, 16), hidden=step * _log_int(rng, 256 // step, 4096 // step),
                inter=step * _log_int(rng, 128 // step, (2048 if bits == 4 else 1024) // step), experts=experts,
                top_k=rng.randint(1, min(8, experts)) if bits == 16 else rng.randint(1, min(6, experts)),
                shared=rng.choice([0, 1, 1, 2]) if bits == 16 else rng.choice([0, 1]), type=rng.choice(["bf16", "bf16", "f16"]),
                bits=bits, group=rng.choice([32, 64, 128]), zeros=bits == 4 and rng.random() < 0.4,
                score=rng.choice(["sigmoid", "softmax"]), bias=rng.random() < 0.5, act=rng.choice(["silu", "silu", "gelu"]))


# ---- inputs ----------------------------------------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    def codes(*shape):
        """Weights in 4 bits, two codes to a byte, and the scales of a matrix of this width."""
        *lead, n, k = shape
        # each code the sum of two numbers of 0..7 and a bit: 0..15, most of them in the middle
        a, b = (torch.randint(0, 256, (*lead, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
                for _ in range(2))
        b = (a & 0x77) + (b & 0x77) + (b >> 3 & 0x11)
        groups = _cdiv(k, case["group"])
        scales = (torch.rand(*lead, n, groups, generator=g, device="cuda") + 0.5) * (0.25 * k ** -0.5)
        z = None
        if case["zeros"]:
            z = torch.randint(5, 11, (*lead, n, groups), generator=g, device="cuda", dtype=torch.uint8)
        return b, scales.to(DTYPES[case["type"]]), z

    def weights(lead, n, k):
        """The experts' matrices [lead, n, k], expert by expert: the numbers in 32 bits are few at a time."""
        if case["bits"] == 4:
            return codes(lead, n, k)
        w = torch.empty(lead, n, k, device="cuda", dtype=DTYPES[case["type"]])
        for part in w.split(16):
            part.copy_(normal(*part.shape, std=k ** -0.5))
        return w

    c, st = case, {"case": dict(case)}
    if c["op"] == "norm":
        rows, hidden, ts, tb = c["rows"], c["hidden"], DTYPES[c["stream"]], DTYPES[c["block"]]
        spread = torch.exp(normal(hidden, std=0.5))  # a stream has a few channels far larger than the rest
        st["state"] = (normal(rows, hidden) * spread).to(ts)
        st["f"] = (normal(rows, hidden) * torch.exp(normal(rows, 1, std=0.3))).to(tb)
        st["w_post"] = 1 + normal(hidden, std=0.1) if c["post"] else None
        st["w_next"] = 1 + normal(hidden, std=0.1)
        shape = {"none": None, "vector": (hidden,), "token": (rows, 1)}[c["gate"]]
        st["gate"] = (0.5 + normal(*shape, std=0.2)).to(tb) if shape else None
        st["scale"] = 0.7
    elif c["op"] == "gated":  # both projections as one product left them
        gu = normal(c["rows"], 2 * c["inter"]) * torch.exp(normal(c["rows"], 1, std=0.5))
        st["gu"] = gu.to(DTYPES[c["type"]])
    elif c["op"] == "int4":
        st["x"] = normal(c["rows"], c["k"]).to(DTYPES[c["type"]])
        st["w"] = codes(c["n"], c["k"])
    elif c["op"] == "weights4":
        st["w"] = (normal(c["n"], c["k"], std=0.02) * torch.exp(normal(c["n"], 1, std=0.3))).to(DTYPES[c["type"]])
    else:
        t, e, h, i = DTYPES[c["type"]], c["experts"], c["hidden"], c["inter"]
        st["x"] = normal(c["rows"], h).to(t)
        st["router"] = normal(e, h, std=1.3 * h ** -0.5).to(t)
        st["bias"] = normal(e, std=0.01) if c["bias"] else None
        st["experts"] = weights(e, i, h), weights(e, i, h), weights(e, h, i)
        s = c["shared"]
        st["shared"] = (weights(s, i, h), weights(s, i, h), weights(s, h, i)) if s else None
    return st


# ---- one pass --------------------------------------------------------------------------------------------


def run(st):
    return {"norm": _norm, "gated": _gated, "int4": _int4, "weights4": _weights4, "routed": _routed}[st["case"]["op"]](st)


def _quantise(y, code, pow2):
    """Codes and scales of blocks of 128 of each row of y (32 bits)."""
    rows, k = y.shape
    kb, most = _cdiv(k, BLOCK), FP8_MAX[code]
    full = torch.zeros(rows, kb * BLOCK, device=y.device)
    full[:, :k] = y
    tiles = full.view(rows, kb, BLOCK)
    amax = tiles.abs().amax(2)
    scale = torch.where(amax == 0, torch.ones_like(amax), (amax / most).clamp_min(2.0 ** -126))
    if pow2:  # up to the next power of two
        m, e = torch.frexp(scale)
        scale = torch.ldexp(torch.ones_like(scale), torch.where(m == 0.5, e - 1, e))
    q = (tiles / scale[:, :, None]).clamp(-most, most).view(rows, -1)[:, :k]
    return q.contiguous().to(FP8[code]), scale


def _norm(st):
    c, f, gate = st["case"], st["f"], st["gate"]
    if own:
        import deepseek_v4_moe_gb300 as m
        return m.block_norm_fp8(st["state"], f, norm_f=st["w_post"], gate=gate, residual_scale=st["scale"],
                                norm_next=st["w_next"], eps=EPS, pow2_scales=c["pow2"], dtype=FP8[c["code"]])
    n = f.float()
    if st["w_post"] is not None:
        n = n * torch.rsqrt(n.square().mean(1, keepdim=True) + EPS) * st["w_post"]
    if gate is not None:
        n = n * gate.float()
    out = (st["state"].float() + st["scale"] * n).to(st["state"].dtype)
    s = out.float()
    return (out, *_quantise(s * torch.rsqrt(s.square().mean(1, keepdim=True) + EPS) * st["w_next"], c["code"], c["pow2"]))


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(GELU_C * (g + 0.044715 * g * g * g)))


def _gated(st):
    c, gu = st["case"], st["gu"]
    g, u = gu[:, :c["inter"]], gu[:, c["inter"]:]
    if own:
        import deepseek_v4_moe_gb300 as m
        return m.gated_quantise(g, u, activation=c["act"], pow2_scales=c["pow2"], dtype=FP8[c["code"]])
    return _quantise(_act(g.float(), c["act"]) * u.float(), c["code"], c["pow2"])


def _values(w, group):
    """What 4-bit weights (codes, scales, zero points) stand for, in 32 bits."""
    codes, scales, zeros = w
    k = codes.shape[-1] * 2
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    z = zeros.float().repeat_interleave(group, -1)[..., :k] if zeros is not None else 8.0
    return (q - z) * scales.float().repeat_interleave(group, -1)[..., :k]


def _int4(st):
    c = st["case"]
    if own:
        import deepseek_v4_moe_gb300 as m
        return m.int4_matmul(st["x"], m.Int4(*st["w"], group=c["group"]))
    return (st["x"].float() @ _values(st["w"], c["group"]).T).to(st["x"].dtype)


def _weights4(st):
    c, w = st["case"], st["w"]
    if own:
        import deepseek_v4_moe_gb300 as m
        q = m.int4_quantise(w, group=c["group"], zero_points=c["zeros"])
        return m.int4_widen(q), q.scales
    n, k = w.shape
    g, least = c["group"], LEAST[c["type"]]
    full = torch.zeros(n, _cdiv(k, g) * g, device=w.device)
    full[:, :k] = w
    full = full.view(n, -1, g)
    if c["zeros"]:
        lo, hi = full.amin(2).clamp_max(0), full.amax(2).clamp_min(0)
        scale = (hi - lo) / 15
    else:
        scale = full.abs().amax(2) / 7
    scale = torch.where(scale == 0, torch.ones_like(scale), scale.clamp_min(least)).to(w.dtype)
    s = scale.float()
    zero = torch.round(-lo / s).clamp(0, 15) if c["zeros"] else torch.full_like(s, 8.0)
    q = (torch.round(full / s[:, :, None]) + zero[:, :, None]).clamp(0 if c["zeros"] else 1, 15)
    return ((q - zero[:, :, None]) * s[:, :, None]).view(n, -1)[:, :k].to(w.dtype).contiguous(), scale


def _routed(st):
    c, x = st["case"], st["x"]
    if own:
        import deepseek_v4_moe_gb300 as m
        four = (lambda w: m.Int4(*w, group=c["group"])) if c["bits"] == 4 else lambda w: w
        return m.routed_ffn(x, st["router"], *(four(w) for w in st["experts"]), top_k=c["top_k"], score=c["score"],
                            bias=st["bias"], shared=tuple(four(w) for w in st["shared"]) if st["shared"] else None,
                            activation=c["act"])
    logits = x.double() @ st["router"].double().T  # 64 bits: two experts' scores may be near one another
    scores = 1 / (1 + torch.exp(-logits)) if c["score"] == "sigmoid" else logits.softmax(1)
    ranked = scores + st["bias"] if st["bias"] is not None else scores
    index = torch.sort(ranked, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
    weight = scores.gather(1, index)
    weight = (weight / weight.sum(1, keepdim=True)).float()

    def rows_of(w, at):  # the matrices of expert at[t] for every token t
        if c["bits"] == 4:
            return _values(tuple(v[at] if v is not None else None for v in w), c["group"])
        return w[at].float()

    def ffn(ws, at):
        gate, up = (torch.bmm(rows_of(w, at), x.float()[:, :, None]) for w in ws[:2])
        return torch.bmm(rows_of(ws[2], at), _act(gate, c["act"]) * up)[:, :, 0]

    y = torch.zeros(x.shape, device=x.device)
    for s in range(c["top_k"]):
        y += weight[:, s, None] * ffn(st["experts"], index[:, s])
    for s in range(c["shared"]):
        y += ffn(st["shared"], torch.full((x.shape[0],), s, device=x.device))
    return y.to(x.dtype), index.int(), weight


# ---- what a pass cannot do without -----------------------------------------------------------------------


def _bytes4(c, n, k):
    return n * k // 2 + n * _cdiv(k, c["group"]) * (3 if c["zeros"] else 2)


def work(case):
    c = case
    if c["op"] == "norm":
        one, blocks = c["rows"] * c["hidden"], c["rows"] * _cdiv(c["hidden"], BLOCK)
        gate = {"none": 0, "vector": c["hidden"], "token": c["rows"]}[c["gate"]] * SIZE[c["block"]]
        norms = 4 * c["hidden"] * (1 + int(c["post"]))
        return {"bytes": one * (2 * SIZE[c["stream"]] + SIZE[c["block"]] + 1) + 4 * blocks + gate + norms,
                "flops": 14 * one}
    if c["op"] == "gated":
        one = c["rows"] * c["inter"]
        return {"bytes": one * (2 * SIZE[c["type"]] + 1) + 4 * c["rows"] * _cdiv(c["inter"], BLOCK), "flops": 12 * one}
    if c["op"] == "int4":
        return {"bytes": _bytes4(c, c["n"], c["k"]) + 2 * c["rows"] * (c["n"] + c["k"]),
                "flops": 2 * c["rows"] * c["n"] * c["k"]}
    if c["op"] == "weights4":  # reads the matrix, writes codes, scales and the widened matrix
        return {"bytes": 4 * c["n"] * c["k"] + _bytes4(c, c["n"], c["k"]), "flops": 6 * c["n"] * c["k"]}
    # routing by near equal chances touches so many of the experts
    touched = c["experts"] * (1 - (1 - c["top_k"] / c["experts"]) ** c["rows"]) + c["shared"]
    h, i = c["hidden"], c["inter"]
    one = 2 * _bytes4(c, i, h) + _bytes4(c, h, i) if c["bits"] == 4 else 6 * h * i
    return {"bytes": int(touched * one) + 2 * c["experts"] * h + 4 * c["rows"] * h,
            "flops": 2 * c["rows"] * (3 * h * i * (c["top_k"] + c["shared"]) + c["experts"] * h)}


# ---- the definitions in 64 bits --------------------------------------------------------------------------


def _codes64(y, code, pow2):
    """Blocks of 128 of y (64 bits) in the format: values over scales, and scales."""
    most = FP8_MAX[code]
    rows, k = y.shape
    amax = torch.nn.functional.pad(y, (0, -k % BLOCK)).unflatten(1, (-1, BLOCK)).abs().amax(2)
    scale = (amax / most).clamp_min(2.0 ** -126)
    if pow2:
        e = torch.floor(torch.log2(scale))
        e = torch.where(torch.exp2(e) < scale, e + 1, e)
        e = torch.where(torch.exp2(e - 1) >= scale, e - 1, e)
        scale = torch.exp2(e)
    scale = torch.where(amax == 0, torch.ones_like(scale), scale)
    v = y / scale[:, torch.arange(k, device="cuda") // BLOCK]
    bits, low = {"e4m3": (3, -6), "e5m2": (2, -14)}[code]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** low))) - bits)
    return (torch.round(v / step) * step).clamp(-most, most), scale


def _wide64(w, group):
    codes, scales, zeros = w
    k = 2 * codes.shape[-1]
    at = torch.arange(k, device="cuda")
    q = ((codes[..., at // 2].int() >> (4 * (at % 2)).int()) & 15).double()
    z = zeros[..., at // group].double() if zeros is not None else 8
    return (q - z) * scales[..., at // group].double()


def exact(case, seed):
    st, c = prepare(case, seed), case

    def act(g):
        if c["act"] == "silu":
            return g * torch.sigmoid(g)
        return g * 0.5 * (1 + ((2 / math.pi) ** 0.5 * (g + 0.044715 * g.pow(3))).tanh())

    if c["op"] == "norm":
        def rms(v, w):
            return v / (v.pow(2).sum(1, keepdim=True) / c["hidden"] + EPS).sqrt() * w

        f = st["f"].double()
        branch = rms(f, st["w_post"].double()) if c["post"] else f
        if st["gate"] is not None:
            branch = branch * st["gate"].double()
        out = st["state"].double() + branch * st["scale"]
        stored = out.to(st["state"].dtype).double()
        return (out, *_codes64(rms(stored, st["w_next"].double()), c["code"], c["pow2"]))
    if c["op"] == "gated":
        g, u = st["gu"].double().split(c["inter"], dim=1)
        return _codes64(act(g) * u, c["code"], c["pow2"])
    if c["op"] == "int4":
        x = st["x"].double()
        parts = zip(*(v.split(8192) if v is not None else [None] * _cdiv(c["n"], 8192) for v in st["w"]))
        return torch.cat([x @ _wide64(w, c["group"]).T for w in parts], 1)
    if c["op"] == "weights4":  # the scales as they are stored: the codes are the quotients by those
        w, k = st["w"].double(), c["k"]
        tiles = torch.nn.functional.pad(w, (0, -k % c["group"])).unflatten(1, (-1, c["group"]))
        lo, hi = tiles.amin(2).clamp_max(0), tiles.amax(2).clamp_min(0)
        scale = (hi - lo) / 15 if c["zeros"] else torch.maximum(hi, -lo) / 7
        scale = torch.where(scale == 0, torch.ones_like(scale), scale.clamp_min(LEAST[c["type"]]))
        stored = scale.to(st["w"].dtype).double()
        zero = torch.round(-lo / stored).clamp(0, 15) if c["zeros"] else torch.full_like(stored, 8)
        at = torch.arange(k, device="cuda") // c["group"]
        q = torch.maximum(torch.round(w / stored[:, at]) + zero[:, at], torch.tensor(0 if c["zeros"] else 1, device="cuda"))
        return (q.clamp_max(15) - zero[:, at]) * stored[:, at], scale
    x = st["x"].double()
    logits = x @ st["router"].double().T
    score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.exp(logits - logits.logsumexp(1, keepdim=True))
    ranked = score + st["bias"].double() if st["bias"] is not None else score
    order = torch.argsort(ranked, dim=1, descending=True, stable=True)[:, :c["top_k"]]
    chosen = torch.gather(score, 1, order)
    chosen = chosen / chosen.sum(1, keepdim=True)

    def matrix(w, e):
        if c["bits"] == 4:
            return _wide64(tuple(v[e] if v is not None else None for v in w), c["group"])
        return w[e].double()

    def block(ws, e, rows):
        g, u, d = (matrix(w, e) for w in ws)
        return (act(rows @ g.T) * (rows @ u.T)) @ d.T

    y = torch.zeros_like(x)
    for e in order.unique().tolist():
        token, slot = (order == e).nonzero(as_tuple=True)
        y.index_add_(0, token, chosen[token, slot, None] * block(st["experts"], e, x[token]))
    for e in range(c["shared"]):
        y += block(st["shared"], e, x)
    return y, order.int(), chosen
