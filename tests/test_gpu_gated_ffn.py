"""gated_ffn and its gradients on the GPU against plain 64-bit arithmetic.

Tolerances, fixed by arithmetic.  e = eps / 2 is the most that a rounding to the operand type is off,
relative.  A result v = sum_k a_k b_k whose a_k were each rounded once is off by sum e_k a_k b_k with
independent |e_k| <= e of mean zero: over 8 e sqrt(sum a_k^2 b_k^2) with a probability below 3e-14 for each
value (Hoeffding).  The tensor cores' f32 sums take 16 products at a time: each such step is off by at most
2^-24 of the magnitudes' sum M (as is its alignment), so a sum over K by (K / 16 + 16) 2^-23 M at most.  The
result's own rounding adds e |v| and half the smallest subnormal."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def half_step(dtype, v):
    f = torch.finfo(dtype)
    return f.eps / 2 * v.abs() + f.smallest_normal * f.eps / 2


def act(name, g):
    if name == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3)))


def sums(k):
    return (k / 16 + 16) * 2.0 ** -23


def make(rows, hidden, inter, dtype, seed=0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*s, std=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * std).to(dtype)

    x, dy = n(rows, hidden + pad)[:, :hidden], n(rows, hidden + pad)[:, :hidden]
    return (x, n(inter, hidden, std=hidden ** -0.5), n(inter, hidden, std=hidden ** -0.5),
            n(hidden, inter, std=inter ** -0.5), dy)


def off(got, ref, tol, what):
    assert got.shape == ref.shape
    err = (got.double() - ref).abs()
    assert (err <= tol).all(), (what, float((err - tol).max()), float((err / tol).max()))


def check(x, wg, wu, wd, dy, name, y, saved, d):
    dt, e = x.dtype, torch.finfo(x.dtype).eps / 2
    rows, hidden = x.shape
    inter = wg.shape[0]
    x, wg, wu, wd, dy = (t.double() for t in (x, wg, wu, wd, dy))
    g, u = x @ wg.T, x @ wu.T
    mg, mu = sums(hidden) * (x.abs() @ wg.abs().T), sums(hidden) * (x.abs() @ wu.abs().T)
    off(saved[0], g, half_step(dt, g) + mg, "g")
    off(saved[1], u, half_step(dt, u) + mu, "u")
    h = act(name, g) * u
    # |act'| <= 1.13, |act(g)| <= |g|
    dh = 1.13 * mg * u.abs() + g.abs() * mu + 2.0 ** -20 * h.abs()
    ref = h @ wd.T
    tol = half_step(dt, ref) + 8 * e * (h ** 2 @ (wd ** 2).T).sqrt() + (sums(inter) * h.abs() + dh) @ wd.abs().T
    off(y, ref, tol, "y")
    if d is None:
        return
    g, u = saved[0].double().requires_grad_(True), saved[1].double().requires_grad_(True)
    hs = act(name, g) * u
    dh = dy @ wd
    dg, du = torch.autograd.grad(hs, (g, u), dh)
    g, u, hs = g.detach(), u.detach(), hs.detach()
    m = sums(hidden) * (dy.abs() @ wd.abs())
    eg, eu = 1.13 * u.abs() * m + 2.0 ** -19 * u.abs() * dh.abs(), g.abs() * m + 2.0 ** -19 * du.abs()
    if "d_x" in d:
        ref = dg @ wg + du @ wu
        tol = (half_step(dt, ref) + 8 * e * (dg ** 2 @ wg ** 2 + du ** 2 @ wu ** 2).sqrt()
               + (sums(2 * inter) * dg.abs() + eg) @ wg.abs() + (sums(2 * inter) * du.abs() + eu) @ wu.abs())
        off(d["d_x"], ref, tol, "d_x")
    if "d_w_gate" in d:
        for k, t, et in (("d_w_gate", dg, eg), ("d_w_up", du, eu)):
            ref = t.T @ x
            tol = half_step(dt, ref) + 8 * e * ((t ** 2).T @ x ** 2).sqrt() + (sums(rows) * t.abs() + et).T @ x.abs()
            off(d[k], ref, tol, k)
        ref = dy.T @ hs
        tol = (half_step(dt, ref) + 8 * e * ((dy ** 2).T @ hs ** 2).sqrt()
               + dy.abs().T @ ((sums(rows) + 2.0 ** -20) * hs.abs()))
        off(d["d_w_down"], ref, tol, "d_w_down")


def run(x, wg, wu, wd, dy, name):
    import deepseek_v4_moe_gb300 as m
    y, saved = m.gated_ffn(x, wg, wu, wd, activation=name, save=True)
    assert torch.equal(m.gated_ffn(x, wg, wu, wd, activation=name), y)
    d = m.gated_ffn_backward(x, wg, wu, wd, saved, dy, activation=name)
    assert m.dense_status() == 0
    return y, saved, d


SIZES = [(1, 8, 8), (1, 64, 64), (2, 72, 136), (3, 128, 128), (4, 1000, 24), (5, 256, 256), (8, 264, 520), (17, 512, 1032),
         (64, 128, 2048), (127, 200, 72), (128, 256, 512), (129, 384, 264), (300, 1000, 1416), (515, 648, 328),
         (1, 4096, 2048), (2, 2048, 4096), (4, 4096, 2048), (70, 4096, 2048), (1500, 512, 384),
         (2049, 1032, 2056), (1100, 4096, 2048)]


@pytest.mark.parametrize("rows,hidden,inter", SIZES)
@pytest.mark.parametrize("dtype,name", [(BF16, "silu"), (F16, "gelu")])
def test_sizes(cuda_lib, rows, hidden, inter, dtype, name):
    t = make(rows, hidden, inter, dtype, seed=rows + hidden + inter, pad=8 * (rows % 3))
    check(*t, name, *run(*t, name))


@pytest.mark.parametrize("dtype,name", [(BF16, "gelu"), (F16, "silu")])
def test_other_types(cuda_lib, dtype, name):
    for rows in (1, 4, 200):
        t = make(rows, 328, 264, dtype, seed=rows)
        check(*t, name, *run(*t, name))


def test_full_size(cuda_lib):
    t = make(4096, 4096, 2048, BF16, seed=1)
    y, saved, d = run(*t, "silu")
    rows = torch.cat([torch.arange(40), torch.randperm(4096, generator=torch.Generator().manual_seed(0))[:200],
                      torch.arange(4060, 4096)]).cuda()
    # rows of y and d_x are computed apart; the weights' gradients take every row
    sub = [t[0][rows], *t[1:4], t[4][rows]]
    check(*sub, "silu", y[rows], [s[rows] for s in saved], {"d_x": d["d_x"][rows]})
    check(*t, "silu", y, saved, d)


def test_only_some_gradients(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    t = make(130, 256, 384, BF16, seed=2)
    y, saved, d = run(*t, "silu")
    x_only = m.gated_ffn_backward(*t[:4], saved, t[4], need_weights=False)
    w_only = m.gated_ffn_backward(*t[:4], saved, t[4], need_x=False)
    assert set(x_only) == {"d_x"} and set(w_only) == {"d_w_gate", "d_w_up", "d_w_down"}
    for k, v in {**x_only, **w_only}.items():
        assert torch.equal(v, d[k])
    with pytest.raises(m.MoeFFNError):
        m.gated_ffn_backward(*t[:4], saved, t[4], need_x=False, need_weights=False)


@pytest.mark.parametrize("rows", [3, 40])
def test_not_finite_stays_in_its_row(cuda_lib, rows):
    import deepseek_v4_moe_gb300 as m
    t = make(rows, 136, 264, BF16, seed=3)
    clean = m.gated_ffn(*t[:4])
    t[0][1, 5] = float("nan")
    t[0][2, 6] = float("inf")
    y = m.gated_ffn(*t[:4])
    keep = [i for i in range(rows) if i not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])
    assert y[1].isnan().all() and not y[2].isfinite().any()


def test_large_gates(cuda_lib):
    # act(g) of gates far out: silu and its derivative saturate without overflow
    import deepseek_v4_moe_gb300 as m
    eye = torch.eye(64, device="cuda", dtype=BF16)
    for rows in (1, 9):
        x = torch.linspace(-300, 300, 64 * rows, device="cuda").view(rows, 64).to(BF16)
        for name in ("silu", "gelu"):
            y, saved = m.gated_ffn(x, eye, eye, eye, activation=name, save=True)
            assert torch.equal(saved[0], x) and torch.equal(saved[1], x)
            ref = act(name, x.double()) * x.double()
            off(y, ref, 3 * half_step(BF16, ref) + 2.0 ** -20 * x.double() ** 2, name)
            d = m.gated_ffn_backward(x, eye, eye, eye, saved, torch.ones_like(x), activation=name)
            assert all(v.isfinite().all() for v in d.values())


def test_against_differences(cuda_lib):
    # the gradients against the 64-bit loss's central differences: <gradient, v> over random directions v;
    # the kernels' gradients are off by about e of each value, so by e sqrt(sum (d v)^2) times a few
    t = make(40, 64, 96, F16, seed=4)
    y, saved, d = run(*t, "silu")
    x, wg, wu, wd, dy = (v.double() for v in t)
    gen = torch.Generator(device="cuda").manual_seed(5)
    base = {"d_x": x, "d_w_gate": wg, "d_w_up": wu, "d_w_down": wd}

    def loss(b):
        return (((act("silu", b["d_x"] @ b["d_w_gate"].T) * (b["d_x"] @ b["d_w_up"].T)) @ b["d_w_down"].T) * dy).sum()

    for k in base:
        v = torch.randn(base[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        diff = (loss({**base, k: base[k] + 1e-5 * v}) - loss({**base, k: base[k] - 1e-5 * v})) / 2e-5
        tol = 40 * 2.0 ** -11 * float((d[k].double() * v).square().sum().sqrt()) + 1e-6 * abs(float(diff))
        assert abs(float((d[k].double() * v).sum() - diff)) <= tol, k


def test_another_stream_and_a_graph(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    for rows in (2, 150):
        t = make(rows, 264, 520, BF16, seed=6)
        y, saved, d = run(*t, "silu")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        y2 = m.gated_ffn(*t[:4], stream=st)
        d2 = m.gated_ffn_backward(*t[:4], saved, t[4], stream=st)
        st.synchronize()
        assert torch.equal(y2, y) and all(torch.equal(d[k], d2[k]) for k in d)
        graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gy, gs = m.gated_ffn(*t[:4], save=True)
            gd = m.gated_ffn_backward(*t[:4], gs, t[4])
        with torch.cuda.graph(other):  # a second graph has a workspace of its own
            oy = m.gated_ffn(*t[:4])
        new = make(rows, 264, 520, BF16, seed=7)
        for a, b in zip(t, new):
            a.copy_(b)
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        check(*t, "silu", gy, gs, gd)
        assert torch.equal(oy, gy)


def test_rows_behind_the_last_stay(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    for rows in (1, 3, 100):
        t = make(rows, 136, 72, BF16, seed=9)
        big = torch.full((rows + 40, 144), 5.0, device="cuda", dtype=BF16)
        y = m.gated_ffn(*t[:4], out=big[:rows, :136])
        assert torch.equal(y, m.gated_ffn(*t[:4]))
        assert (big[rows:] == 5).all() and (big[:, 136:] == 5).all()


def test_a_wait_that_runs_out_is_reported(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    for size in ((200, 256, 256), (4096, 2048, 2048)):  # single CTAs, and pairs
        t = make(*size, BF16, seed=10)
        good = m.gated_ffn(*t[:4])
        assert m.dense_status() == 0
        assert cuda_lib.moe_ffn_dense_fault_injection(1, 20000) == 0
        try:
            m.gated_ffn(*t[:4])
            assert m.dense_status() == 8
        finally:
            cuda_lib.moe_ffn_dense_fault_injection(0, 0)
        assert torch.equal(m.gated_ffn(*t[:4]), good)
        assert m.dense_status() == 0


def test_refusals(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    x, wg, wu, wd, dy = make(6, 64, 72, BF16)
    for bad in (lambda: m.gated_ffn(x.float(), wg, wu, wd), lambda: m.gated_ffn(x, wg, wu, wd.T),
                lambda: m.gated_ffn(x, wg.half(), wu, wd), lambda: m.gated_ffn(x, wg, wu[:64], wd),
                lambda: m.gated_ffn(x, wg, wu, wd, activation="relu"), lambda: m.gated_ffn(x.cpu(), wg, wu, wd),
                lambda: m.gated_ffn(x, wg, wu, wd, out=dy.float()), lambda: m.gated_ffn(x.T, wg, wu, wd)):
        with pytest.raises(ValueError):
            bad()
    wide = torch.zeros(6, 70, device="cuda", dtype=BF16)
    y, saved = m.gated_ffn(x, wg, wu, wd, save=True)
    for code, bad in ((-4, lambda: m.gated_ffn(x[:0], wg, wu, wd)), (-2, lambda: m.gated_ffn(wide[:, :64], wg, wu, wd)),
                      (-2, lambda: m.gated_ffn(x[:, :60].contiguous(), wg[:, :60].contiguous(), wu[:, :60].contiguous(),
                                               wd[:60].contiguous())),
                      (-11, lambda: m.gated_ffn(torch.zeros(6 * 64 + 1, device="cuda", dtype=BF16)[1:].view(6, 64), wg, wu, wd)),
                      (-7, lambda: m.gated_ffn(x, wg, wu, wd, out=x))):
        with pytest.raises(m.MoeFFNError) as e:
            bad()
        assert e.value.code == code
    with pytest.raises(ValueError):
        m.gated_ffn_backward(x, wg, wu, wd, (saved[0], saved[1][:, :64]), dy)
