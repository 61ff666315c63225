"""The dense sublayer's C entry points without a GPU: the argument checks answer before any CUDA call."""
import ctypes

import pytest

from deepseek_v4_moe_gb300 import _lib

A = 1 << 20  # fake addresses, a MiB apart: never dereferenced, the checks that answer run first


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def _norm(**kw):
    base = dict(rows=4, hidden=256, stream_type=_lib.TYPE_F32, block_type=_lib.TYPE_BF16, gate_type=_lib.TYPE_BF16,
                gate_kind=_lib.GATE_NONE, rows_per_gate=1, residual_scale=1.0, eps=1e-6, state=A, ld_state=256,
                f=2 * A, ld_f=256, gate=None, norm_f=3 * A, norm_next=4 * A, out=5 * A, ld_out=256, y=6 * A, ld_y=256)
    base.update(kw)
    return _lib.MoeFfnBlockNormArgs(**base)


NORM_REFUSED = [
    (dict(rows=0), _lib.ERR_ROWS_ZERO), (dict(rows=-1), _lib.ERR_ROWS_RANGE), (dict(hidden=0), _lib.ERR_BAD_CONFIG),
    (dict(hidden=8193), _lib.ERR_BAD_CONFIG), (dict(stream_type=_lib.TYPE_F16), _lib.ERR_BAD_CONFIG),
    (dict(block_type=7), _lib.ERR_BAD_CONFIG), (dict(eps=-1.0), _lib.ERR_BAD_CONFIG),
    (dict(eps=float("nan")), _lib.ERR_BAD_CONFIG), (dict(state=None), _lib.ERR_NULL_PTR),
    (dict(f=None, norm_f=None, out=None, norm_next=None, y=None), _lib.ERR_NULL_PTR),
    (dict(f=None, out=None), _lib.ERR_BAD_CONFIG),            # norm_f without f
    (dict(ld_state=255), _lib.ERR_BAD_CONFIG), (dict(ld_f=0), _lib.ERR_BAD_CONFIG),
    (dict(ld_out=255), _lib.ERR_BAD_CONFIG), (dict(ld_y=255), _lib.ERR_BAD_CONFIG),
    (dict(out=None), _lib.ERR_NULL_PTR), (dict(y=None), _lib.ERR_NULL_PTR),
    (dict(norm_next=None), _lib.ERR_NULL_PTR),                # y without norm_next
    (dict(gate_kind=1), _lib.ERR_NULL_PTR), (dict(gate_kind=9, gate=7 * A), _lib.ERR_BAD_CONFIG),
    (dict(gate_kind=1, gate=7 * A, rows_per_gate=0), _lib.ERR_BAD_CONFIG),
    (dict(gate_kind=2, gate=7 * A, gate_type=_lib.TYPE_F16), _lib.ERR_BAD_CONFIG),
    (dict(gate_kind=2, gate=7 * A + 1), _lib.ERR_ALIGNMENT), (dict(state=A + 2), _lib.ERR_ALIGNMENT),
    (dict(y=6 * A + 1), _lib.ERR_ALIGNMENT), (dict(out=A + 4), _lib.ERR_ALIAS),
    (dict(out=A, ld_out=260), _lib.ERR_ALIAS),                # the state's memory at another stride
    (dict(y=2 * A), _lib.ERR_ALIAS), (dict(y=5 * A + 512), _lib.ERR_ALIAS), (dict(out=4 * A), _lib.ERR_ALIAS),
    (dict(gate_kind=1, gate=5 * A + 16), _lib.ERR_ALIAS),
]


@pytest.mark.parametrize("kw,code", NORM_REFUSED)
def test_block_norm_refuses(lib, kw, code):
    assert lib.moe_ffn_block_norm(ctypes.byref(_norm(**kw)), None) == code, lib.moe_ffn_last_error(None)


def _grads(**kw):
    base = dict(d_out=8 * A, ld_d_out=256, d_y=9 * A, ld_d_y=256, d_state=10 * A, ld_d_state=256, d_f=11 * A,
                ld_d_f=256, d_gate=None, d_norm_f=12 * A, d_norm_next=13 * A, workspace=14 * A, workspace_bytes=0)
    base.update(kw)
    return _lib.MoeFfnBlockNormGrads(**base)


@pytest.mark.parametrize("kw,gkw,code", [
    ({}, dict(d_state=None), _lib.ERR_NULL_PTR), ({}, dict(d_f=None), _lib.ERR_NULL_PTR),
    ({}, dict(d_y=None), _lib.ERR_NULL_PTR), (dict(norm_next=None), {}, _lib.ERR_BAD_CONFIG),
    ({}, dict(d_gate=15 * A), _lib.ERR_BAD_CONFIG), (dict(norm_f=None), {}, _lib.ERR_BAD_CONFIG),
    ({}, dict(ld_d_f=100), _lib.ERR_BAD_CONFIG), ({}, dict(ld_d_out=255), _lib.ERR_BAD_CONFIG),
    ({}, dict(d_state=10 * A + 1), _lib.ERR_ALIGNMENT), ({}, dict(workspace=14 * A + 8), _lib.ERR_ALIGNMENT),
    ({}, dict(d_state=A), _lib.ERR_ALIAS), ({}, dict(d_f=9 * A), _lib.ERR_ALIAS),
    ({}, dict(d_f=8 * A), _lib.ERR_ALIAS), ({}, dict(d_norm_f=13 * A + 4), _lib.ERR_ALIAS),
    ({}, dict(workspace=10 * A, workspace_bytes=64), _lib.ERR_ALIAS),
])
def test_block_norm_backward_refuses(lib, kw, gkw, code):
    rc = lib.moe_ffn_block_norm_backward(ctypes.byref(_norm(**kw)), ctypes.byref(_grads(**gkw)), None)
    assert rc == code, lib.moe_ffn_last_error(None)


def test_block_norm_null(lib):
    assert lib.moe_ffn_block_norm(None, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_block_norm_backward(ctypes.byref(_norm()), None, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_block_norm_workspace(None, None) == _lib.ERR_NULL_PTR


def _gated(**kw):
    base = dict(rows=4, hidden=256, inter=64, type=_lib.TYPE_BF16, activation=0, x=A, ld_x=256, w_gate=2 * A, w_up=3 * A,
                w_down=4 * A, y=5 * A, ld_y=256, gate=6 * A, up=7 * A, d_y=8 * A, ld_d_y=256, d_x=9 * A, ld_d_x=256,
                d_w_gate=10 * A, d_w_up=11 * A, d_w_down=12 * A, workspace=13 * A, workspace_bytes=1536)
    base.update(kw)
    return _lib.MoeFfnGatedArgs(**base)


BOTH_REFUSED = [
    (dict(rows=0), _lib.ERR_ROWS_ZERO), (dict(rows=-3), _lib.ERR_ROWS_RANGE), (dict(rows=(1 << 24) + 1), _lib.ERR_ROWS_RANGE),
    (dict(hidden=0), _lib.ERR_BAD_CONFIG), (dict(hidden=252), _lib.ERR_BAD_CONFIG), (dict(inter=65544), _lib.ERR_BAD_CONFIG),
    (dict(type=_lib.TYPE_F32), _lib.ERR_BAD_CONFIG), (dict(activation=2), _lib.ERR_BAD_CONFIG),
    (dict(x=None), _lib.ERR_NULL_PTR), (dict(w_up=None), _lib.ERR_NULL_PTR), (dict(workspace=None), _lib.ERR_NULL_PTR),
    (dict(ld_x=248), _lib.ERR_BAD_CONFIG), (dict(ld_x=257), _lib.ERR_BAD_CONFIG), (dict(ld_x=1 << 40), _lib.ERR_BAD_CONFIG),
    (dict(x=A + 8), _lib.ERR_ALIGNMENT), (dict(w_down=4 * A + 2), _lib.ERR_ALIGNMENT), (dict(up=None), _lib.ERR_NULL_PTR),
    (dict(gate=6 * A + 4), _lib.ERR_ALIGNMENT), (dict(workspace_bytes=100), _lib.ERR_NO_MEMORY),
    (dict(workspace=A), _lib.ERR_ALIAS),
]


@pytest.mark.parametrize("kw,code", BOTH_REFUSED + [
    (dict(y=None), _lib.ERR_NULL_PTR), (dict(ld_y=100), _lib.ERR_BAD_CONFIG), (dict(y=A), _lib.ERR_ALIAS),
    (dict(gate=5 * A), _lib.ERR_ALIAS), (dict(y=13 * A + 16), _lib.ERR_ALIAS)])
def test_gated_forward_refuses(lib, kw, code):
    assert lib.moe_ffn_gated_forward(ctypes.byref(_gated(**kw)), None) == code, lib.moe_ffn_last_error(None)


@pytest.mark.parametrize("kw,code", BOTH_REFUSED + [
    (dict(d_y=None), _lib.ERR_NULL_PTR), (dict(d_w_up=None), _lib.ERR_NULL_PTR), (dict(d_x=8 * A), _lib.ERR_ALIAS),
    (dict(d_x=None, d_w_gate=None, d_w_up=None, d_w_down=None), _lib.ERR_NULL_PTR),
    (dict(d_w_gate=11 * A), _lib.ERR_ALIAS), (dict(d_x=6 * A), _lib.ERR_ALIAS), (dict(ld_d_x=128), _lib.ERR_BAD_CONFIG),
    (dict(workspace_bytes=1535), _lib.ERR_NO_MEMORY)])
def test_gated_backward_refuses(lib, kw, code):
    assert lib.moe_ffn_gated_backward(ctypes.byref(_gated(**kw)), None) == code, lib.moe_ffn_last_error(None)


def test_gated_workspace(lib):
    assert lib.moe_ffn_gated_workspace(ctypes.byref(_gated()), 0) == 4 * 64 * 2
    assert lib.moe_ffn_gated_workspace(ctypes.byref(_gated()), 1) == 4 * 64 * 2 * 3
    assert lib.moe_ffn_gated_workspace(ctypes.byref(_gated(rows=0)), 1) == _lib.ERR_ROWS_ZERO
    assert lib.moe_ffn_gated_workspace(None, 1) == _lib.ERR_NULL_PTR


def _matmul(**kw):
    base = dict(rows=4, n=200, k=256, a_type=0, b_type=0, out_type=_lib.TYPE_BF16, a=A, ld_a=256, a_scale=2 * A, b=3 * A,
                ld_b=256, b_scale=4 * A, out=5 * A, ld_out=200)
    base.update(kw)
    return _lib.MoeFfnFp8MatmulArgs(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), _lib.ERR_ROWS_ZERO), (dict(rows=-1), _lib.ERR_ROWS_RANGE), (dict(n=0), _lib.ERR_BAD_CONFIG),
    (dict(k=0), _lib.ERR_BAD_CONFIG), (dict(k=40), _lib.ERR_BAD_CONFIG), (dict(a_type=2), _lib.ERR_BAD_CONFIG),
    (dict(b_type=-1), _lib.ERR_BAD_CONFIG), (dict(out_type=3), _lib.ERR_BAD_CONFIG), (dict(a=None), _lib.ERR_NULL_PTR),
    (dict(b_scale=None), _lib.ERR_NULL_PTR), (dict(ld_a=264), _lib.ERR_BAD_CONFIG), (dict(ld_b=240), _lib.ERR_BAD_CONFIG),
    (dict(ld_out=199), _lib.ERR_BAD_CONFIG), (dict(a=A + 8), _lib.ERR_ALIGNMENT), (dict(b_scale=4 * A + 2), _lib.ERR_ALIGNMENT),
    (dict(out=5 * A + 1), _lib.ERR_ALIGNMENT), (dict(out=A), _lib.ERR_ALIAS), (dict(out=2 * A), _lib.ERR_ALIAS)])
def test_fp8_matmul_refuses(lib, kw, code):
    assert lib.moe_ffn_fp8_matmul(ctypes.byref(_matmul(**kw)), None) == code, lib.moe_ffn_last_error(None)


def _quantise(**kw):
    base = dict(rows=4, k=256, type=_lib.TYPE_BF16, code_type=0, block_rows=1, pow2=0, x=A, ld_x=256, codes=2 * A,
                ld_codes=256, scales=3 * A)
    base.update(kw)
    return _lib.MoeFfnFp8QuantiseArgs(**base)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=0), _lib.ERR_ROWS_ZERO), (dict(rows=-1), _lib.ERR_ROWS_RANGE), (dict(k=0), _lib.ERR_BAD_CONFIG),
    (dict(type=5), _lib.ERR_BAD_CONFIG), (dict(code_type=2), _lib.ERR_BAD_CONFIG), (dict(block_rows=64), _lib.ERR_BAD_CONFIG),
    (dict(x=None), _lib.ERR_NULL_PTR), (dict(scales=None), _lib.ERR_NULL_PTR), (dict(ld_x=255), _lib.ERR_BAD_CONFIG),
    (dict(ld_codes=255), _lib.ERR_BAD_CONFIG), (dict(x=A + 1), _lib.ERR_ALIGNMENT), (dict(scales=3 * A + 2), _lib.ERR_ALIGNMENT),
    (dict(codes=A), _lib.ERR_ALIAS), (dict(scales=2 * A + 16), _lib.ERR_ALIAS)])
def test_fp8_quantise_refuses(lib, kw, code):
    assert lib.moe_ffn_fp8_quantise(ctypes.byref(_quantise(**kw)), None) == code, lib.moe_ffn_last_error(None)


def test_fp8_null(lib):
    assert lib.moe_ffn_fp8_matmul(None, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_fp8_quantise(None, None) == _lib.ERR_NULL_PTR


# ---- column ranges of one tensor are apart, though their rows lie between one another ----

@pytest.mark.parametrize("kw", [
    dict(), dict(state=A + 1024, out=A), dict(y=A + 4096 - 512), dict(state=A + 4096 + 2048, out=A, y=A + 1024)])
def test_column_ranges_of_one_tensor(lib, kw):
    # bytes: state f32 of 1024 in a pitch of 4096, out behind it, y of 512 behind that; nothing refuses them, and
    # the call ends where its device would have to be looked up
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not memory")
    args = dict(rows=4, ld_state=1024, state=A, out=A + 1024, ld_out=1024, y=A + 2048, ld_y=2048)
    args.update(kw)
    assert lib.moe_ffn_block_norm(ctypes.byref(_norm(**args)), None) in (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED)


@pytest.mark.parametrize("kw", [
    dict(out=A + 1020), dict(out=A + 4), dict(out=A + 4096 - 1020), dict(out=A + 4096 + 4), dict(out=A - 4),
    dict(y=A + 1022), dict(y=A + 2046), dict(y=A + 4096 - 510)])
def test_column_ranges_that_overlap(lib, kw):
    args = dict(rows=4, ld_state=1024, state=A, out=A + 1024, ld_out=1024, y=A + 2048, ld_y=2048)
    args.update(kw)
    assert lib.moe_ffn_block_norm(ctypes.byref(_norm(**args)), None) == _lib.ERR_ALIAS


def test_block_norm_rows_past_the_limit(lib):
    for rows in (2 ** 30 + 1, 2 ** 31 - 1):
        assert lib.moe_ffn_block_norm(ctypes.byref(_norm(rows=rows)), None) == _lib.ERR_ROWS_RANGE
        assert lib.moe_ffn_block_norm_workspace(ctypes.byref(_norm(rows=rows)), ctypes.byref(_grads())) == _lib.ERR_ROWS_RANGE
