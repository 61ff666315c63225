"""The dense sublayer's operators where a documented call reaches a limit: every tile of the matrix products,
tensors that are parts of one another's storage, offsets past 2^32, groups of rows that do not divide the
rows, rows whose norm's cube leaves f32, waits that run out in the backward pass, first calls under capture,
calls from several threads, and errors.  References and tolerances are those of the operators' own tests."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import test_gpu_dense_norm as tn
import test_gpu_fp8 as t8
import test_gpu_gated_ffn as tg

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# between them they take every tile of every product on 152 SMs: 32 to 256 columns, by one CTA, a pair, or
# clusters of two and four that share k
TILES = [(5, 32, 32), (5, 2016, 2736), (394, 2664, 208), (5, 3088, 2416), (1796, 1400, 656), (5552, 840, 104),
         (676, 1608, 3688), (1321, 32, 32), (812, 3864, 2000), (4966, 456, 960), (1027, 3720, 1984),
         (1035, 4056, 1720), (2662, 3032, 1216), (541, 4488, 6736)]
TILES8 = [(47, 133, 160), (8, 4935, 176), (4964, 1, 3328), (17, 20, 2944), (3233, 2621, 16), (4958, 200, 2656),
          (539, 3903, 1152), (2619, 1376, 2208)]


@pytest.mark.parametrize("rows,hidden,inter", TILES)
def test_every_tile_of_the_gated_block(cuda_lib, rows, hidden, inter):
    dtype, name = ((BF16, "silu"), (F16, "gelu"))[rows % 2]
    t = tg.make(rows, hidden, inter, dtype, seed=rows)
    tg.check(*t, name, *tg.run(*t, name))


@pytest.mark.parametrize("rows,n,k", TILES8)
@pytest.mark.parametrize("out", [BF16, F32])
def test_every_tile_of_the_fp8_product(cuda_lib, rows, n, k, out):
    import deepseek_v4_moe_gb300 as m
    gen = torch.Generator(device="cuda").manual_seed(rows)
    a, sa = t8.operand(rows, k, 1, E4, gen)
    b, sb = t8.operand(n, k, 128, E5, gen)
    t8.check(a, sa, b, sb, m.fp8_matmul(a, sa, b, sb, out_dtype=out))
    assert m.dense_status() == 0


@pytest.mark.parametrize("rows", [3, 150])
def test_column_ranges_of_one_tensor(cuda_lib, rows):
    """Inputs and outputs side by side in one tensor, which holds NaN wherever nobody should read."""
    import deepseek_v4_moe_gb300 as m
    h = 256

    def part(t, at, cols=h):
        return t[:, at:at + cols]

    c = tn.make(rows, h, F32, F32, "vector", True, True, seed=rows)
    t = torch.full((rows + 2, 5 * h + 64), float("nan"), device="cuda")
    state, f, out, y = (part(t[1:-1], at) for at in (0, h + 32, 2 * h + 32, 4 * h + 64))
    state.copy_(c["state"]), f.copy_(c["f"])
    kw = {k: c[k] for k in ("norm_f", "gate", "residual_scale", "norm_next", "eps")}
    want = m.block_norm(c["state"], c["f"], **kw)
    got = m.block_norm(state, f, out=out, y=y, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(state, c["state"])
    assert t[0].isnan().all() and t[-1].isnan().all() and t[:, h:h + 32].isnan().all()

    x, wg, wu, wd, _ = tg.make(rows, h, 136, BF16, seed=rows)
    t = torch.full((rows + 2, 3 * h), float("nan"), device="cuda", dtype=BF16)
    a, b = part(t[1:-1], h), part(t[1:-1], 0)
    a.copy_(x)
    assert torch.equal(m.gated_ffn(a, wg, wu, wd, out=b), m.gated_ffn(x, wg, wu, wd))
    assert torch.equal(a, x) and t[0].isnan().all() and t[-1].isnan().all() and t[:, 2 * h:].isnan().all()
    with pytest.raises(m.MoeFFNError) as e:
        m.gated_ffn(a, wg, wu, wd, out=part(t[1:-1], 8))
    assert e.value.code == -7
    assert torch.equal(m.gated_ffn(x, wg, wg, wd), m.gated_ffn(x, wg, wg.clone(), wd))  # one tensor twice


def far(rows, cols, dtype):
    """A [rows, cols] tensor whose last row begins past 2^31 elements and 2^32 bytes."""
    size = torch.empty(0, dtype=dtype).element_size()
    ld = ((1 << 32) // size // (rows - 1) // 64 + 1) * 64
    return torch.empty((rows - 1) * ld + cols, device="cuda", dtype=dtype).as_strided((rows, cols), (ld, 1))


@pytest.mark.parametrize("rows", [2, 3, 6])
def test_offsets_past_32_bits(cuda_lib, rows):
    import deepseek_v4_moe_gb300 as m
    c = tn.make(rows, 264, BF16, BF16, "token", True, True, seed=rows)
    kw = {k: c[k] for k in ("norm_f", "gate", "residual_scale", "norm_next", "eps")}
    want = m.block_norm(c["state"], c["f"], **kw)
    w = {k: far(rows, 264, BF16).copy_(c[k]) for k in ("state", "f")}
    assert w["f"].stride(0) * (rows - 1) >= 1 << 31
    out, y = m.block_norm(w["state"], w["f"], out=far(rows, 264, BF16), y=far(rows, 264, BF16), **kw)
    assert torch.equal(out, want[0]) and torch.equal(y, want[1])
    d = m.block_norm_backward(want[0], c["f"], d_out=c["d_out"], d_y=c["d_y"], **kw)
    e = m.block_norm_backward(out, w["f"], d_out=far(rows, 264, BF16).copy_(c["d_out"]), d_y=y.copy_(c["d_y"]), **kw)
    assert all(torch.equal(d[k], e[k]) for k in d)
    del w, out, y

    x, wg, wu, wd, dy = tg.make(rows, 264, 136, BF16, seed=rows)
    fx = far(rows, 264, BF16).copy_(x)
    want, saved = m.gated_ffn(x, wg, wu, wd, save=True)
    assert torch.equal(m.gated_ffn(fx, wg, wu, wd, out=far(rows, 264, BF16)), want)
    d = m.gated_ffn_backward(x, wg, wu, wd, saved, dy)
    e = m.gated_ffn_backward(fx, wg, wu, wd, saved, far(rows, 264, BF16).copy_(dy))
    assert all(torch.equal(d[k], e[k]) for k in d)

    codes, scales = m.fp8_quantise(x)
    fc, fs = m.fp8_quantise(fx)
    assert torch.equal(codes.view(torch.uint8), fc.view(torch.uint8)) and torch.equal(scales, fs)
    k = 256
    a, b = codes[:, :k], m.fp8_quantise(wg[:, :k].contiguous(), block_rows=128)
    fa = far(rows, k, E4)
    fa.view(torch.uint8).copy_(a.view(torch.uint8))
    sa = scales[:, :2].contiguous()
    a = a.contiguous()
    assert torch.equal(m.fp8_matmul(fa, sa, *b, out=far(rows, 136, BF16)), m.fp8_matmul(a, sa, *b))


@pytest.mark.parametrize("rows,per", [(24, 7), (5000, 1700), (5, 9), (5000, 4999)])
def test_gate_groups_that_do_not_divide_the_rows(cuda_lib, rows, per):
    import deepseek_v4_moe_gb300 as m
    from deepseek_v4_moe_gb300 import _lib
    h, n = 1024, -(-rows // per)
    c = tn.make(rows, h, BF16, BF16, "full", True, True, seed=rows)
    gate = c["gate"][:n].contiguous()
    c["gate"] = gate.repeat_interleave(per, 0)[:rows].contiguous()
    out, y = torch.empty_like(c["state"]), torch.empty_like(c["state"])
    a = _lib.MoeFfnBlockNormArgs(rows=rows, hidden=h, stream_type=1, block_type=1, gate_type=1, gate_kind=1, rows_per_gate=per,
                                 residual_scale=c["residual_scale"], eps=c["eps"], state=c["state"].data_ptr(), ld_state=h,
                                 f=c["f"].data_ptr(), ld_f=h, gate=gate.data_ptr(), norm_f=c["norm_f"].data_ptr(),
                                 norm_next=c["norm_next"].data_ptr(), out=out.data_ptr(), ld_out=h, y=y.data_ptr(), ld_y=h)
    st = torch.cuda.current_stream().cuda_stream
    assert cuda_lib.moe_ffn_block_norm(ctypes.byref(a), st) == 0
    tn.check_forward(c, out, y)
    d = {k: torch.full_like(v, float("nan")) for k, v in dict(d_state=out, d_f=out, d_gate=gate, d_norm_f=c["norm_f"],
                                                               d_norm_next=c["norm_next"]).items()}
    a.state = out.data_ptr()
    g = _lib.MoeFfnBlockNormGrads(d_out=c["d_out"].data_ptr(), ld_d_out=h, d_y=c["d_y"].data_ptr(), ld_d_y=h,
                                  ld_d_state=h, ld_d_f=h, **{k: v.data_ptr() for k, v in d.items()})
    need = cuda_lib.moe_ffn_block_norm_workspace(ctypes.byref(a), ctypes.byref(g))
    ws = torch.empty(max(need, 1), device="cuda", dtype=torch.uint8)
    g.workspace, g.workspace_bytes = ws.data_ptr(), need
    assert cuda_lib.moe_ffn_block_norm_backward(ctypes.byref(a), ctypes.byref(g), st) == 0
    torch.cuda.synchronize()
    ref = tn.reference_grads(c, out)
    pad = n * per - rows
    ref["d_gate"] = tuple(torch.cat([v, v.new_zeros(pad, h)]).view(n, per, h).sum(1) for v in ref["d_gate"])
    for k, (v, mag) in ref.items():
        terms = rows if k not in ("d_state", "d_f") else 0
        tol = tn.half_step(d[k].dtype, v) + (160 + terms) * tn.U * mag
        assert ((d[k].double() - v).abs() <= tol).all(), k


@pytest.mark.parametrize("size", [1e14, 1e-14])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("hidden", [1000, 1001])
def test_norms_whose_cube_leaves_f32(cuda_lib, size, post, hidden):
    """Rows of 1e14 and 1e-14 are normal f32 values, and so are their norms and gradients."""
    c = tn.make(9, hidden, F32, F32, "vector", post, not post, seed=1)
    c["eps"] = 0.0
    c["f"] = c["f"] * size
    if not post:
        c["state"] = c["state"] * size
        c["d_out"] = c["d_out"] / size
    out, y, d = tn.both(c)
    tn.check_forward(c, out, y)
    tn.check_backward(c, out, d)


@pytest.mark.parametrize("rows,hidden,inter", [(5, 3088, 2416), (300, 520, 264), (2662, 3032, 1216)])
def test_a_wait_that_runs_out_in_the_backward_pass(cuda_lib, rows, hidden, inter):
    """CTA 0 of each of the three kernels gives up after 20 ms; the next call finds everything in order."""
    import deepseek_v4_moe_gb300 as m
    t = tg.make(rows, hidden, inter, BF16, seed=2)
    y, saved, good = tg.run(*t, "silu")
    assert cuda_lib.moe_ffn_dense_fault_injection(1, 20000) == 0
    try:
        m.gated_ffn_backward(*t[:4], saved, t[4])
        assert m.dense_status() == 8
    finally:
        cuda_lib.moe_ffn_dense_fault_injection(0, 0)
    d = m.gated_ffn_backward(*t[:4], saved, t[4])
    assert m.dense_status() == 0 and all(torch.equal(d[k], good[k]) for k in good)


def test_status_under_capture_is_refused(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    x, wg, wu, wd, _ = tg.make(40, 64, 72, BF16)
    want = m.gated_ffn(x, wg, wu, wd)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = m.gated_ffn(x, wg, wu, wd)
        with pytest.raises(m.MoeFFNError) as e:
            m.dense_status()
    assert e.value.code == -10
    got.zero_()
    g.replay()
    assert torch.equal(got, want) and m.dense_status() == 0


FIRST = """
import torch, deepseek_v4_moe_gb300 as m
torch.manual_seed(0)
B = torch.bfloat16
x, wg, wu, wd = (torch.randn(*s, device="cuda").to(B) for s in ((40, 256), (320, 256), (320, 256), (256, 320)))
w = torch.ones(256, device="cuda")
g = torch.cuda.CUDAGraph()
def step():
    s, y = m.block_norm(x, norm_next=w)
    f, saved = m.gated_ffn(y, wg, wu, wd, save=True)
    q = m.fp8_matmul(*m.fp8_quantise(f), *m.fp8_quantise(wg, block_rows=128))
    return [f, q, *m.gated_ffn_backward(y, wg, wu, wd, saved, f).values(),
            *m.block_norm_backward(s, norm_next=w, d_y=f).values(), m.gated_ffn(x[:2], wg, wu, wd)]
with torch.cuda.graph(g):
    out = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step())) and m.dense_status() == 0
print("same")
"""


def test_first_calls_of_a_process_under_capture(cuda_lib):
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr


def test_calls_from_several_threads(cuda_lib):
    import deepseek_v4_moe_gb300 as m
    sizes = [(2, 512, 264), (70, 512, 264), (300, 520, 1032), (700, 1024, 512)]

    def job(i):
        x, wg, wu, wd, dy = tg.make(*sizes[i], BF16, seed=i)
        w = torch.ones(sizes[i][1], device="cuda")

        def step():
            s, y = m.block_norm(x, norm_next=w)
            f, saved = m.gated_ffn(y, wg, wu, wd, save=True)
            d = m.gated_ffn_backward(y, wg, wu, wd, saved, dy)
            return [f, *d.values(), *m.block_norm_backward(s, norm_next=w, d_y=d["d_x"], d_out=dy).values()]
        return step

    jobs = [job(i) for i in range(len(sizes))]
    want = [j() for j in jobs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(20):
                    got = jobs[i]()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                        bad.append(i)
                    m.dense_status()
        except Exception as e:  # a thread's failure is the test's
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(sizes))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad


def test_memory_that_is_not_there(cuda_lib):
    """The saved projections of 2^22 rows of 65536 values take 512 GiB each: PyTorch's own error, and the next
    call works."""
    import deepseek_v4_moe_gb300 as m
    x = torch.zeros(1 << 22, 8, device="cuda", dtype=BF16)
    wg = torch.zeros(65536, 8, device="cuda", dtype=BF16)
    wd = torch.zeros(8, 65536, device="cuda", dtype=BF16)
    with pytest.raises(torch.cuda.OutOfMemoryError):
        m.gated_ffn(x, wg, wg, wd, save=True)
    assert not m.gated_ffn(x[:64], wg, wg, wd).any() and m.dense_status() == 0


def test_what_comes_before_and_after_on_the_stream(cuda_lib):
    """Kernels start while the one before them ends: each still reads what copies, fills, kernels and other
    streams' work before it wrote, and is done before what follows it writes."""
    import deepseek_v4_moe_gb300 as m
    rows, h = 2048, 2048
    host = [torch.randn(rows, h, generator=torch.Generator().manual_seed(i)).to(BF16).pin_memory() for i in range(3)]
    _, wg, wu, wd, _ = tg.make(1, h, 512, BF16, seed=1)
    w = torch.ones(h, device="cuda")

    def ops(x):
        s, y = m.block_norm(x, norm_next=w)
        few = m.gated_ffn(x[:2], wg, wu, wd)
        f = m.gated_ffn(y, wg, wu, wd)
        q = m.fp8_quantise(f)
        return [few, f, *q, m.fp8_matmul(*q, *m.fp8_quantise(wg, block_rows=128)),
                *m.block_norm_backward(s, norm_next=w, d_y=f).values()]

    want = [[t.clone() for t in ops(t.cuda())] for t in host]
    torch.cuda.synchronize()
    x, x2 = torch.empty(2, rows, h, device="cuda", dtype=BF16).unbind()
    side = torch.cuda.Stream()

    def chain():
        got = []
        for i, t in enumerate(host):
            x.copy_(t, non_blocking=True)          # a copy before
            got.append((i, ops(x)))
            x.zero_()                              # a fill after
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):          # a kernel of another stream before, joined by an event
                x2.copy_(t, non_blocking=True)
                x2.mul_(1.0)
            torch.cuda.current_stream().wait_stream(side)
            got.append((i, ops(x2)))
            x2.fill_(float("nan"))
            x2.copy_(x)                            # zeros, by a kernel
            x.copy_(host[(i + 1) % 3], non_blocking=True)
            got.append(((i + 1) % 3, ops(x)))
        return got

    def check(got):
        torch.cuda.synchronize()
        for i, g in got:
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(g, want[i])), i

    for _ in range(3):
        check(chain())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    for _ in range(3):
        for _, t in got:
            for v in t:
                v.view(torch.uint8).zero_()
        g.replay()
        check(got)
    assert m.dense_status() == 0


# the same for the backward pass's products in one launch and in two (both ways of every size), and the rest
MORE_TILES = [(5, 32, 2088), (5, 5544, 392), (5, 2544, 2904), (665, 264, 920), (937, 1752, 136), (2491, 984, 648),
              (3394, 5376, 32), (1583, 32, 3752), (756, 32, 72), (1045, 2896, 584), (555, 1936, 2472), (4245, 936, 1472),
              (804, 856, 4184), (513, 1888, 6128), (513, 1976, 7168)]


@pytest.mark.parametrize("rows,hidden,inter", MORE_TILES)
def test_gradients_together_and_apart(cuda_lib, rows, hidden, inter):
    import deepseek_v4_moe_gb300 as m
    dtype, name = ((BF16, "silu"), (F16, "gelu"))[(rows + inter // 8) % 2]
    t = tg.make(rows, hidden, inter, dtype, seed=rows)
    y, saved, d = tg.run(*t, name)
    tg.check(*t, name, y, saved, d)
    apart = m.gated_ffn_backward(*t[:4], saved, t[4], activation=name, need_weights=False)
    apart.update(m.gated_ffn_backward(*t[:4], saved, t[4], activation=name, need_x=False))
    tg.check(*t, name, y, saved, apart)
    assert m.dense_status() == 0


@pytest.mark.parametrize("rows", [1, 4, 8, 40])
def test_weights_that_the_kernel_before_makes(cuda_lib, rows):
    """Each weight of the gated block comes from a kernel just before it on the stream, after others that
    started early: nothing is read before it is written."""
    import deepseek_v4_moe_gb300 as m
    h, inter = 512, 256
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, wg, wu, _, _ = tg.make(rows, h, inter, BF16, seed=rows)
    pairs = [(m.fp8_quantise(torch.randn(h, 4096, generator=gen, device="cuda") / 64),
              m.fp8_quantise(torch.randn(inter, 4096, generator=gen, device="cuda"), block_rows=128)) for _ in range(3)]
    made = [m.fp8_matmul(*a, *b) for a, b in pairs]
    want = [m.gated_ffn(x, wg, wu, w) for w in made]
    torch.cuda.synchronize()
    wd = torch.empty(h, inter, device="cuda", dtype=BF16)

    def chain():
        got = []
        for i in range(12):
            (a, b), w = pairs[i % 3], made[(i + 1) % 3]
            m.fp8_matmul(*a, *b, out=wd)
            got.append((i % 3, m.gated_ffn(x, wg, wu, wd)))
            m.block_norm(w, norm_next=torch.ones(inter, device="cuda"), y=wd)
            wd.copy_(w)
            m.fp8_quantise(x)
            got.append(((i + 1) % 3, m.gated_ffn(x, wg, wu, wd)))
        return got

    for _ in range(5):
        got = chain()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i]) for i, y in got)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = chain()
    for _ in range(5):
        wd.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want[i]) for i, y in got)
    assert m.dense_status() == 0


@pytest.mark.parametrize("ts,tb", [(F32, F32), (F32, BF16), (BF16, BF16)])
@pytest.mark.parametrize("rows,hidden", [(3, 8192), (700, 8192), (310, 8184), (5, 8190)])
@pytest.mark.parametrize("gate", ["vector", "group", "token"])
def test_the_longest_rows(cuda_lib, ts, tb, rows, hidden, gate):
    """Rows whose ring leaves the weights no shared memory, or holds one row."""
    if gate == "group" and rows % max(1, rows // 3):
        rows += -rows % 3
    c = tn.make(rows, hidden, ts, tb, gate, True, True, seed=hidden)
    if gate == "group":
        c["gate"] = c["gate"][:3].contiguous()
    out, y, d = tn.both(c)
    tn.check_forward(c, out, y)
    tn.check_backward(c, out, d)


@pytest.mark.parametrize("rows,hidden,inter", [(9, 2048, 1024), (100, 1024, 2048), (127, 4096, 512)])
def test_only_the_weights_gradients_of_few_rows(cuda_lib, rows, hidden, inter):
    import deepseek_v4_moe_gb300 as m
    t = tg.make(rows, hidden, inter, BF16, seed=rows)
    y, saved, d = tg.run(*t, "silu")
    d = m.gated_ffn_backward(*t[:4], saved, t[4], need_x=False)
    assert set(d) == {"d_w_gate", "d_w_up", "d_w_down"}
    tg.check(*t, "silu", y, saved, d)
