"""block_norm and its gradients on the GPU against plain 64-bit arithmetic.

Tolerances, fixed by arithmetic: a stored value is off by half a step of its type (eps / 2 relative,
and half the smallest subnormal); the f32 work before that by a multiple of u = 2^-24 of the sum of the
magnitudes that enter it (M below): a row sum of n terms in the kernel's order, 8 in a thread, then a
butterfly over at most 1024 threads, is off by at most (8 + 10) u relative when its terms are of one
sign, its rsqrt by half of that and 2 ulp; products and sums around it add a few u.  K = 64 covers a
value that passes one such norm, 160 one that passes two; a sum over rows adds one u for each row."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


def half_step(dtype, v):
    f = torch.finfo(dtype)
    return f.eps / 2 * v.abs() + f.smallest_normal * f.eps / 2


def rms(v, eps):
    return 1 / (v.square().mean(1, keepdim=True) + eps).sqrt()


def gate_rows(gate, rows, hidden):
    if gate is None:
        return torch.ones(1, 1, dtype=torch.float64, device="cuda")
    g = gate.double()
    if tuple(g.shape) == (rows, 1):
        return g
    if g.dim() == 1:
        return g[None]
    return g.repeat_interleave(rows // g.shape[0], 0)


def make(rows, hidden, ts, tb, gate, post, nxt, seed=0, gate_dtype=None):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*s, std=1.0):
        return torch.randn(*s, generator=g, device="cuda") * std

    shape = {"none": None, "vector": (hidden,), "token": (rows, 1), "full": (rows, hidden),
             "group": (max(1, rows // 3), hidden)}[gate]
    return dict(state=n(rows, hidden).to(ts), f=n(rows, hidden, std=3.0).to(tb),
                norm_f=1 + n(hidden, std=0.2) if post else None, norm_next=1 + n(hidden, std=0.2) if nxt else None,
                gate=n(*shape).to(gate_dtype or tb) if shape else None, residual_scale=0.6, eps=1e-6,
                d_out=n(rows, hidden).to(ts), d_y=n(rows, hidden).to(tb) if nxt else None)


def check_forward(c, out, y):
    f, s, al = c["f"].double(), c["state"].double(), c["residual_scale"]
    rows, hidden = f.shape
    n = f * (rms(f, c["eps"]) * c["norm_f"].double() if c["norm_f"] is not None else 1.0)
    branch = al * gate_rows(c["gate"], rows, hidden) * n
    ref = s + branch
    tol = half_step(out.dtype, ref) + 64 * U * (s.abs() + branch.abs())
    assert ((out.double() - ref).abs() <= tol).all(), "out"
    if c["norm_next"] is not None:
        o = out.double()  # the norm takes the stream as stored
        ref = o * rms(o, c["eps"]) * c["norm_next"].double()
        assert ((y.double() - ref).abs() <= half_step(y.dtype, ref) + 64 * U * ref.abs()).all(), "y"
    else:
        assert y is None


def reference_grads(c, out):
    """{name: (gradient, magnitude of what was added up)} in 64 bits."""
    f, s, al, eps = c["f"].double(), out.double(), c["residual_scale"], c["eps"]
    rows, hidden = f.shape
    go = c["d_out"].double()
    ds, m_ds = go, go.abs()
    r = {}
    if c["norm_next"] is not None:
        gy, w, rs = c["d_y"].double(), c["norm_next"].double(), rms(s, eps)
        ds = go + rs * (gy * w - s * rs ** 2 * (gy * w * s).mean(1, keepdim=True))
        m_ds = go.abs() + rs * ((gy * w).abs() + s.abs() * rs ** 2 * (gy * w * s).abs().mean(1, keepdim=True))
        t = gy * s * rs
        r["d_norm_next"] = (t.sum(0), t.abs().sum(0))
    r["d_state"] = (ds, m_ds)
    g = gate_rows(c["gate"], rows, hidden)
    rf = rms(f, eps) if c["norm_f"] is not None else 1.0
    w = c["norm_f"].double() if c["norm_f"] is not None else 1.0
    if c["gate"] is not None:
        t, m = al * f * rf * w * ds, (al * f * rf * w).abs() * m_ds
        shape = tuple(c["gate"].shape)
        if shape == (rows, 1):
            r["d_gate"] = (t.sum(1, keepdim=True), m.sum(1, keepdim=True))
        elif shape == (hidden,):
            r["d_gate"] = (t.sum(0), m.sum(0))
        else:
            k = rows // shape[0]
            r["d_gate"] = (t.view(shape[0], k, hidden).sum(1), m.view(shape[0], k, hidden).sum(1))
    dn, m = al * g * ds, (al * g).abs() * m_ds
    if c["norm_f"] is not None:
        r["d_norm_f"] = ((dn * f * rf).sum(0), (m * (f * rf).abs()).sum(0))
        dw, m = dn * w, m * w.abs()
        r["d_f"] = (rf * (dw - f * rf ** 2 * (dw * f).mean(1, keepdim=True)),
                    rf * (m + f.abs() * rf ** 2 * (m * f.abs()).mean(1, keepdim=True)))
    else:
        r["d_f"] = (dn, m)
    return r


def check_backward(c, out, d):
    ref = reference_grads(c, out)
    assert set(d) == set(ref)
    rows, hidden = c["f"].shape
    for k, (v, m) in ref.items():
        terms = rows if k in ("d_norm_f", "d_norm_next") or (k == "d_gate" and d[k].shape[0] != rows) else 0
        if k == "d_gate" and tuple(d[k].shape) == (rows, 1):
            terms = 18
        tol = half_step(d[k].dtype, v) + (160 + terms) * U * m
        err = (d[k].double() - v).abs()
        assert (err <= tol).all(), (k, float((err - tol).max()), float((err / tol).max()))


def both(c):
    import deepseek_v4_moe_gb300 as m
    kw = {k: c[k] for k in ("norm_f", "gate", "residual_scale", "norm_next", "eps")}
    out, y = m.block_norm(c["state"], c["f"], **kw)
    d = m.block_norm_backward(out, c["f"], d_out=c["d_out"], d_y=c["d_y"], **kw)
    return out, y, d


TYPES = [(F32, F32), (F32, BF16), (F32, F16), (BF16, BF16), (F16, F16)]


@pytest.mark.parametrize("ts,tb", TYPES)
@pytest.mark.parametrize("rows,hidden", [(1, 4096), (5, 1), (3, 7), (33, 64), (2, 255), (130, 1000), (77, 1001),
                                         (700, 128), (9, 4104), (3, 8192), (2, 8191)])
def test_sizes_and_types(cuda_lib, ts, tb, rows, hidden):
    gate = ["vector", "token", "full", "none"][(rows + hidden) % 4]
    c = make(rows, hidden, ts, tb, gate, True, True, seed=rows * 10000 + hidden)
    out, y, d = both(c)
    check_forward(c, out, y)
    check_backward(c, out, d)


@pytest.mark.parametrize("gate", ["none", "vector", "token", "full", "group"])
@pytest.mark.parametrize("post,nxt", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("rows", [1, 6, 900])
def test_gates_and_norms(cuda_lib, gate, post, nxt, rows):
    for gate_dtype in (None, F32):
        c = make(rows, 392, F32, BF16, gate, post, nxt, seed=rows, gate_dtype=gate_dtype)
        out, y, d = both(c)
        check_forward(c, out, y)
        check_backward(c, out, d)


def test_many_rows_sum_over_workers_and_chunks(cuda_lib):
    # more rows than the grid has groups; gate rows whose chunks several workers share
    for gate in ("vector", "group"):
        c = make(5001, 512, BF16, BF16, gate, True, True, seed=3)
        if gate == "group":
            c["gate"] = c["gate"][:3].contiguous()
        out, y, d = both(c)
        check_forward(c, out, y)
        check_backward(c, out, d)


def test_norm_before_only(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    g = torch.Generator(device="cuda").manual_seed(5)
    s = torch.randn(19, 640, generator=g, device="cuda")
    w = torch.rand(640, generator=g, device="cuda") + 0.5
    out, y = m.block_norm(s, norm_next=w, block_dtype=BF16)
    assert out is s
    ref = s.double() * rms(s.double(), 1e-6) * w.double()
    assert ((y.double() - ref).abs() <= half_step(BF16, ref) + 64 * U * ref.abs()).all()
    gy = torch.randn(19, 640, generator=g, device="cuda").to(BF16)
    d = m.block_norm_backward(s, norm_next=w, d_y=gy)
    assert set(d) == {"d_state", "d_norm_next"}
    sd = s.double().requires_grad_(True)
    wd = w.double().requires_grad_(True)
    ds, dw = torch.autograd.grad(sd * rms(sd, 1e-6) * wd, (sd, wd), gy.double())
    mag = rms(s.double(), 1e-6) * ((gy.double() * w).abs() + s.abs().double() * rms(s.double(), 1e-6) ** 2
                                   * (gy.double() * w * s).abs().mean(1, keepdim=True))
    assert ((d["d_state"].double() - ds).abs() <= half_step(F32, ds) + 160 * U * mag).all()
    assert torch.allclose(d["d_norm_next"].double(), dw, rtol=0, atol=float(200 * U * (gy.double() * s).abs().sum(0).max()))


def test_against_differences(cuda_lib):
    # <gradient, direction> against the 64-bit loss's central difference along it: the difference is
    # off by O(h^2) of the loss's third derivative, small at h = 1e-4 against 1e-5 relative to the
    # sum of magnitudes
    c = make(7, 96, F32, F32, "vector", True, True, seed=11)
    out, y, d = both(c)
    g = torch.Generator(device="cuda").manual_seed(12)
    names = {"state": "d_state", "f": "d_f", "gate": "d_gate", "norm_f": "d_norm_f", "norm_next": "d_norm_next"}
    base = {k: c[k].double() for k in names}

    def loss(v):
        n = v["f"] * rms(v["f"], c["eps"]) * v["norm_f"]
        s = v["state"] + c["residual_scale"] * v["gate"] * n
        yy = s * rms(s, c["eps"]) * v["norm_next"]
        return (s * c["d_out"].double()).sum() + (yy * c["d_y"].double()).sum()

    for k, dk in names.items():
        v = torch.randn(base[k].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-4
        diff = (loss({**base, k: base[k] + h * v}) - loss({**base, k: base[k] - h * v})) / (2 * h)
        got = (d[dk].double() * v).sum()
        assert abs(float(got - diff)) <= 1e-5 * float((d[dk].double() * v).abs().sum()), k


@pytest.mark.parametrize("wide", [True, False])
def test_strided_rows_in_place_and_untouched_rows(cuda_lib, wide):
    import deepseek_v4_moe_gb300 as m
    pad = 8 if wide else 3
    c = make(21, 264, BF16, BF16, "token", True, True, seed=8)
    big = {k: torch.full((25, 264 + pad), 7.0, dtype=BF16, device="cuda") for k in ("state", "f", "y")}
    big["state"][:21, :264], big["f"][:21, :264] = c["state"], c["f"]
    s, f, y = (big[k][:21, :264] for k in ("state", "f", "y"))
    kw = {k: c[k] for k in ("norm_f", "gate", "residual_scale", "norm_next", "eps")}
    out, yy = m.block_norm(s, f, out=s, y=y, **kw)
    assert out.data_ptr() == s.data_ptr()
    check_forward(c, out, yy)
    for k in ("state", "y"):  # what lies beside and behind the rows stays
        assert (big[k][21:] == 7).all() and (big[k][:, 264:] == 7).all()


def test_zero_rows_and_values_that_are_not_finite(cuda_lib):
    c = make(6, 300, F32, BF16, "token", True, True, seed=9)
    c["f"][1] = 0
    c["state"][2] = 0
    c["f"][2] = 0          # a row of nothing at all
    c["f"][4, 17] = float("inf")
    c["state"][5, 3] = float("nan")
    out, y, d = both(c)
    keep = [0, 1, 2, 3]
    sub = {k: (v[keep] if torch.is_tensor(v) and v.dim() == 2 else v) for k, v in c.items()}
    check_forward(sub, out[keep], y[keep])
    assert (out[2] == 0).all() and (y[2] == 0).all()
    ref = reference_grads(sub, out[keep])
    for k in ("d_state", "d_f", "d_gate"):
        v, mm = ref[k]
        assert ((d[k][keep].double() - v).abs() <= half_step(d[k].dtype, v) + 200 * U * mm).all(), k
    assert y[5].isnan().all() and not y[keep].isnan().any()
    assert not out[4].isfinite().all()


def test_same_bits_again_on_another_stream_and_in_a_graph(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    c = make(700, 1032, F32, BF16, "vector", True, True, seed=21)
    kw = {k: c[k] for k in ("norm_f", "gate", "residual_scale", "norm_next", "eps")}
    out, y, d = both(c)
    again = both(c)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    o2, y2 = m.block_norm(c["state"], c["f"], stream=st, **kw)
    d2 = m.block_norm_backward(o2, c["f"], d_out=c["d_out"], d_y=c["d_y"], stream=st, **kw)
    st.synchronize()
    for a, b in ((again[0], out), (again[1], y), (o2, out), (y2, y)):
        assert torch.equal(a, b)
    for k in d:
        assert torch.equal(d[k], again[2][k]) and torch.equal(d[k], d2[k])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go, gy = m.block_norm(c["state"], c["f"], **kw)
        gd = m.block_norm_backward(go, c["f"], d_out=c["d_out"], d_y=c["d_y"], **kw)
    new = make(700, 1032, F32, BF16, "vector", True, True, seed=22)
    for k in ("state", "f", "d_out", "d_y", "gate", "norm_f", "norm_next"):
        c[k].copy_(new[k])
    graph.replay()
    torch.cuda.synchronize()
    check_forward(c, go, gy)
    check_backward(c, go, gd)


def test_python_refuses(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    c = make(4, 64, F32, BF16, "none", True, True)
    s, f, w = c["state"], c["f"], c["norm_next"]
    for bad in (lambda: m.block_norm(s, f[:3], norm_next=w), lambda: m.block_norm(s.cpu(), f.cpu()),
                lambda: m.block_norm(s.to(F16), f), lambda: m.block_norm(s, f, norm_next=w.to(BF16)),
                lambda: m.block_norm(s, f, gate=torch.ones(3, 64, device="cuda")),
                lambda: m.block_norm(s, f, gate=torch.ones(4, device="cuda")),
                lambda: m.block_norm(s.T, f), lambda: m.block_norm(s, norm_f=w, norm_next=w),
                lambda: m.block_norm(s, f, y=f), lambda: m.block_norm_backward(s),
                lambda: m.block_norm_backward(s, f, norm_next=w), lambda: m.block_norm(s.long(), f)):
        with pytest.raises(ValueError):
            bad()
    for code, bad in ((-4, lambda: m.block_norm(s[:0], f[:0])), (-7, lambda: m.block_norm(f, f, out=f[:, :])),
                      (-2, lambda: m.block_norm(s, f, eps=float("nan"))),
                      (-2, lambda: m.block_norm(torch.zeros(1, 9000, device="cuda"), torch.zeros(1, 9000, device="cuda")))):
        if code == -7:
            g = f.clone()
            bad = lambda: m.block_norm(g, f, out=f)  # noqa: E731
        with pytest.raises(m.MoeFFNError) as e:
            bad()
        assert e.value.code == code
