"""The C entry points for a few rows and for operands of the FP8 product, without a GPU: the argument checks answer before
any CUDA call."""
import ctypes

import pytest

from deepseek_v4_moe_gb300 import _lib

A = 1 << 24  # fake addresses, 16 MiB apart: never dereferenced, the checks that answer run first
BF16, F16, F32 = _lib.TYPE_BF16, _lib.TYPE_F16, _lib.TYPE_F32


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def said(lib):
    return lib.moe_ffn_last_error(None)


# ---- operands of the FP8 product ----

def _out(**kw):
    return _lib.MoeFfnFp8Out(**{**dict(code_type=0, pow2=0, codes=7 * A, ld_codes=256, scales=8 * A), **kw})


def _norm(**kw):
    base = dict(rows=4, hidden=256, stream_type=F32, block_type=BF16, gate_type=BF16, gate_kind=_lib.GATE_NONE,
                rows_per_gate=1, residual_scale=1.0, eps=1e-6, state=A, ld_state=256, f=2 * A, ld_f=256, gate=None,
                norm_f=3 * A, norm_next=4 * A, out=5 * A, ld_out=256, y=None, ld_y=0)
    return _lib.MoeFfnBlockNormArgs(**{**base, **kw})


OUT_REFUSED = [(dict(code_type=2), _lib.ERR_BAD_CONFIG), (dict(codes=None), _lib.ERR_NULL_PTR), (dict(scales=None), _lib.ERR_NULL_PTR),
               (dict(ld_codes=255), _lib.ERR_BAD_CONFIG), (dict(scales=8 * A + 2), _lib.ERR_ALIGNMENT),
               (dict(scales=7 * A + 16), _lib.ERR_ALIAS)]


@pytest.mark.parametrize("kw,okw,code", [({}, o, c) for o, c in OUT_REFUSED] + [
    (dict(y=6 * A, ld_y=256), {}, _lib.ERR_BAD_CONFIG), (dict(norm_next=None), {}, _lib.ERR_NULL_PTR),
    (dict(rows=0), {}, _lib.ERR_ROWS_ZERO), (dict(hidden=8193), {}, _lib.ERR_BAD_CONFIG), (dict(eps=-1.0), {}, _lib.ERR_BAD_CONFIG),
    ({}, dict(codes=A), _lib.ERR_ALIAS), ({}, dict(codes=5 * A), _lib.ERR_ALIAS), ({}, dict(scales=4 * A), _lib.ERR_ALIAS)])
def test_block_norm_fp8_refuses(lib, kw, okw, code):
    assert lib.moe_ffn_block_norm_fp8(ctypes.byref(_norm(**kw)), ctypes.byref(_out(**okw)), None) == code, said(lib)


def _gated(**kw):
    base = dict(rows=4, columns=256, type=BF16, activation=0, gate=A, ld_gate=512, up=A + 512, ld_up=512)
    return _lib.MoeFfnGatedQuantiseArgs(**{**base, **kw})


@pytest.mark.parametrize("kw,okw,code", [({}, o, c) for o, c in OUT_REFUSED] + [
    (dict(rows=0), {}, _lib.ERR_ROWS_ZERO), (dict(rows=(1 << 24) + 1), {}, _lib.ERR_ROWS_RANGE), (dict(columns=0), {}, _lib.ERR_BAD_CONFIG),
    (dict(columns=(1 << 20) + 8), {}, _lib.ERR_BAD_CONFIG), (dict(type=F32), {}, _lib.ERR_BAD_CONFIG),
    (dict(activation=2), {}, _lib.ERR_BAD_CONFIG), (dict(gate=None), {}, _lib.ERR_NULL_PTR), (dict(up=A + 1), {}, _lib.ERR_ALIGNMENT),
    (dict(ld_up=255), {}, _lib.ERR_BAD_CONFIG), ({}, dict(codes=A + 64), _lib.ERR_ALIAS)])
def test_gated_quantise_refuses(lib, kw, okw, code):
    assert lib.moe_ffn_gated_quantise(ctypes.byref(_gated(**kw)), ctypes.byref(_out(**okw)), None) == code, said(lib)


# ---- weights in 4 bits ----

def _weights(**kw):
    base = dict(n=64, k=256, group=128, scale_type=BF16, codes=2 * A, scales=3 * A, zeros=4 * A)
    return _lib.MoeFfnInt4WeightsArgs(**{**base, **kw})


WEIGHTS_REFUSED = [(dict(n=0), _lib.ERR_BAD_CONFIG), (dict(n=(1 << 24) + 1), _lib.ERR_BAD_CONFIG), (dict(k=0), _lib.ERR_BAD_CONFIG),
                   (dict(k=48), _lib.ERR_BAD_CONFIG), (dict(k=(1 << 20) + 32), _lib.ERR_BAD_CONFIG), (dict(group=16), _lib.ERR_BAD_CONFIG),
                   (dict(group=96), _lib.ERR_BAD_CONFIG), (dict(scale_type=F32), _lib.ERR_BAD_CONFIG), (dict(codes=None), _lib.ERR_NULL_PTR),
                   (dict(scales=None), _lib.ERR_NULL_PTR), (dict(codes=2 * A + 8), _lib.ERR_ALIGNMENT),
                   (dict(scales=3 * A + 2), _lib.ERR_ALIGNMENT), (dict(zeros=4 * A + 1), _lib.ERR_ALIGNMENT)]


@pytest.mark.parametrize("kw,w,kind,ld,code", [(kw, A, F32, 256, c) for kw, c in WEIGHTS_REFUSED] + [
    ({}, None, F32, 256, _lib.ERR_NULL_PTR), ({}, A, 5, 256, _lib.ERR_BAD_CONFIG), ({}, A, BF16, 248, _lib.ERR_BAD_CONFIG),
    ({}, A, BF16, 260, _lib.ERR_BAD_CONFIG), ({}, A + 16, F32, 256, _lib.ERR_ALIGNMENT), ({}, A + 8, BF16, 256, _lib.ERR_ALIGNMENT),
    (dict(codes=A), A, BF16, 256, _lib.ERR_ALIAS), (dict(scales=2 * A), A, BF16, 256, _lib.ERR_ALIAS),
    (dict(zeros=3 * A), A, BF16, 256, _lib.ERR_ALIAS)])
def test_int4_quantise_refuses(lib, kw, w, kind, ld, code):
    assert lib.moe_ffn_int4_quantise(ctypes.byref(_weights(**kw)), w, kind, ld, None) == code, said(lib)


@pytest.mark.parametrize("kw,out,ld,code", [(kw, A, 256, c) for kw, c in WEIGHTS_REFUSED] + [
    ({}, None, 256, _lib.ERR_NULL_PTR), ({}, A, 248, _lib.ERR_BAD_CONFIG), ({}, A, 260, _lib.ERR_BAD_CONFIG),
    ({}, A + 8, 256, _lib.ERR_ALIGNMENT), (dict(codes=A), A, 256, _lib.ERR_ALIAS), (dict(scales=A + 64), A, 256, _lib.ERR_ALIAS)])
def test_int4_widen_refuses(lib, kw, out, ld, code):
    assert lib.moe_ffn_int4_widen(ctypes.byref(_weights(**kw)), out, ld, None) == code, said(lib)


def _matmul(**kw):
    base = dict(rows=20, n=64, k=256, type=BF16, group=128, x=A, ld_x=256, codes=2 * A, scales=3 * A, zeros=4 * A, out=5 * A,
                ld_out=64, workspace=6 * A, workspace_bytes=1 << 20)
    return _lib.MoeFfnInt4MatmulArgs(**{**base, **kw})


SIZES_REFUSED = [(dict(rows=0), _lib.ERR_ROWS_ZERO), (dict(rows=-1), _lib.ERR_ROWS_RANGE), (dict(rows=(1 << 16) + 1), _lib.ERR_ROWS_RANGE),
                 (dict(type=F32), _lib.ERR_BAD_CONFIG), (dict(n=0), _lib.ERR_BAD_CONFIG), (dict(k=40), _lib.ERR_BAD_CONFIG),
                 (dict(group=48), _lib.ERR_BAD_CONFIG)]


@pytest.mark.parametrize("kw,code", SIZES_REFUSED + [
    (dict(x=None), _lib.ERR_NULL_PTR), (dict(codes=None), _lib.ERR_NULL_PTR), (dict(scales=None), _lib.ERR_NULL_PTR),
    (dict(out=None), _lib.ERR_NULL_PTR), (dict(ld_x=248), _lib.ERR_BAD_CONFIG), (dict(ld_x=260), _lib.ERR_BAD_CONFIG),
    (dict(ld_out=63), _lib.ERR_BAD_CONFIG), (dict(x=A + 8), _lib.ERR_ALIGNMENT), (dict(out=5 * A + 1), _lib.ERR_ALIGNMENT),
    (dict(codes=2 * A + 8), _lib.ERR_ALIGNMENT), (dict(workspace=6 * A + 16), _lib.ERR_ALIGNMENT), (dict(out=A), _lib.ERR_ALIAS),
    (dict(out=2 * A + 64), _lib.ERR_ALIAS), (dict(out=4 * A), _lib.ERR_ALIAS), (dict(workspace=5 * A), _lib.ERR_ALIAS),
    (dict(workspace=A + 1024), _lib.ERR_ALIAS)])
def test_int4_matmul_refuses(lib, kw, code):
    assert lib.moe_ffn_int4_matmul(ctypes.byref(_matmul(**kw)), None) == code, said(lib)


@pytest.mark.parametrize("kw,code", SIZES_REFUSED)
def test_int4_matmul_workspace_refuses(lib, kw, code):
    assert lib.moe_ffn_int4_matmul_workspace(ctypes.byref(_matmul(**kw))) == code, said(lib)


# (rows, n, k, group) and whether x is split into planes first
FORMS = [(1, 64, 64, 32, False), (8, 4096, 4096, 128, False), (16, 4096, 4096, 64, False), (1, 8193, 4096, 128, True),
         (8, 8191, 4096, 128, False), (1, 8193, 4096, 64, False), (8, 10000, 6752, 64, True), (16, 40, 8192, 64, True),
         (8, 40, 8192, 64, False), (16, 40, 8160, 128, False), (16, 129280, 4096, 32, False), (17, 32, 32, 32, True),
         (17, 20000, 512, 32, False), (17, 20000, 512, 64, True), (33, 2999, 64, 32, True), (33, 3001, 64, 32, False),
         (65536, 300, 256, 128, True)]


@pytest.mark.parametrize("rows,n,k,group,planes", FORMS)
def test_int4_matmul_workspace(lib, rows, n, k, group, planes):
    for kind, count in ((BF16, 2), (F16, 3)):
        size = lib.moe_ffn_int4_matmul_workspace(ctypes.byref(_matmul(rows=rows, n=n, k=k, group=group, type=kind, x=None)))
        assert (size >= rows * count * k) if planes else size == 0


def test_null(lib):
    assert lib.moe_ffn_int4_matmul(None, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_int4_matmul_workspace(None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_int4_quantise(None, A, 0, 8, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_int4_widen(None, A, 8, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_routed_forward(None, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_routed_workspace(None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_gated_quantise(None, ctypes.byref(_out()), None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_gated_quantise(ctypes.byref(_gated()), None, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_block_norm_fp8(ctypes.byref(_norm()), None, None) == _lib.ERR_NULL_PTR
    assert lib.moe_ffn_block_norm_fp8(None, ctypes.byref(_out()), None) == _lib.ERR_NULL_PTR


# ---- the routed layer ----

M = _lib.MoeFfnMatrices


def _routed(bits=16, **kw):
    scales = bits == 4
    mats = {n: M(w=(10 + i) * A, scales=(20 + i) * A if scales else None, zeros=None)
            for i, n in enumerate(("gate", "up", "down", "shared_gate", "shared_up", "shared_down"))}
    base = dict(rows=4, hidden=256, inter=64, experts=8, top_k=2, shared=1, type=BF16, router_type=F32, bits=bits, group=64,
                score=0, normalise=1, activation=0, route_scale=1.0, x=A, ld_x=256, router=2 * A, bias=3 * A, y=4 * A, ld_y=256,
                indices=5 * A, weights=6 * A, workspace=7 * A, workspace_bytes=1 << 22, **mats)
    return _lib.MoeFfnRoutedArgs(**{**base, **kw})


LAYER_REFUSED = [
    (dict(rows=0), _lib.ERR_ROWS_ZERO), (dict(rows=-1), _lib.ERR_ROWS_RANGE), (dict(rows=33), _lib.ERR_ROWS_RANGE),
    (dict(bits=8), _lib.ERR_BAD_CONFIG), (dict(hidden=0), _lib.ERR_BAD_CONFIG), (dict(hidden=252), _lib.ERR_BAD_CONFIG),
    (dict(inter=65544), _lib.ERR_BAD_CONFIG), (dict(experts=0), _lib.ERR_BAD_CONFIG), (dict(experts=513), _lib.ERR_BAD_CONFIG),
    (dict(top_k=0), _lib.ERR_BAD_CONFIG), (dict(top_k=9), _lib.ERR_BAD_CONFIG), (dict(experts=1), _lib.ERR_BAD_CONFIG),
    (dict(shared=-1), _lib.ERR_BAD_CONFIG), (dict(shared=9), _lib.ERR_BAD_CONFIG), (dict(type=F32), _lib.ERR_BAD_CONFIG),
    (dict(router_type=F16), _lib.ERR_BAD_CONFIG), (dict(score=2), _lib.ERR_BAD_CONFIG), (dict(activation=2), _lib.ERR_BAD_CONFIG)]


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("kw,code", LAYER_REFUSED + [
    (dict(x=None), _lib.ERR_NULL_PTR), (dict(router=None), _lib.ERR_NULL_PTR), (dict(y=None), _lib.ERR_NULL_PTR),
    (dict(workspace=None), _lib.ERR_NULL_PTR), (dict(ld_x=248), _lib.ERR_BAD_CONFIG), (dict(ld_x=252), _lib.ERR_BAD_CONFIG),
    (dict(ld_y=255), _lib.ERR_BAD_CONFIG), (dict(x=A + 8), _lib.ERR_ALIGNMENT), (dict(router=2 * A + 16), _lib.ERR_ALIGNMENT),
    (dict(bias=3 * A + 2), _lib.ERR_ALIGNMENT), (dict(indices=5 * A + 2), _lib.ERR_ALIGNMENT), (dict(y=4 * A + 1), _lib.ERR_ALIGNMENT),
    (dict(workspace=7 * A + 8), _lib.ERR_ALIGNMENT), (dict(workspace_bytes=128), _lib.ERR_NO_MEMORY), (dict(y=A), _lib.ERR_ALIAS),
    (dict(weights=5 * A + 4), _lib.ERR_ALIAS), (dict(workspace=10 * A), _lib.ERR_ALIAS), (dict(workspace=4 * A), _lib.ERR_ALIAS),
    (dict(shared=0), _lib.ERR_BAD_CONFIG), (dict(gate=M(w=None)), _lib.ERR_NULL_PTR)])
def test_routed_refuses(lib, bits, kw, code):
    assert lib.moe_ffn_routed_forward(ctypes.byref(_routed(**{"bits": bits, **kw})), None) == code, said(lib)


def test_routed_refuses_by_bits(lib):
    def rc(bits, **kw):
        return lib.moe_ffn_routed_forward(ctypes.byref(_routed(bits, **kw)), None)
    assert rc(4, group=96) == _lib.ERR_BAD_CONFIG and rc(4, hidden=264, ld_x=264) == _lib.ERR_BAD_CONFIG
    assert rc(4, up=M(w=11 * A)) == _lib.ERR_NULL_PTR                                                 # no scales
    assert rc(4, up=M(w=11 * A, scales=21 * A, zeros=31 * A)) == _lib.ERR_BAD_CONFIG                  # zero points of one projection
    assert rc(16, up=M(w=11 * A, scales=21 * A)) == _lib.ERR_BAD_CONFIG
    assert rc(16, down=M(w=12 * A + 8)) == _lib.ERR_ALIGNMENT and rc(4, down=M(w=12 * A + 8, scales=22 * A)) == _lib.ERR_ALIGNMENT
    assert rc(4, shared_up=M(w=14 * A, scales=24 * A + 4)) == _lib.ERR_ALIGNMENT


@pytest.mark.parametrize("kw,code", LAYER_REFUSED)
def test_routed_workspace_refuses(lib, kw, code):
    assert lib.moe_ffn_routed_workspace(ctypes.byref(_routed(**kw))) == code, said(lib)


@pytest.mark.parametrize("bits", [4, 16])
def test_routed_workspace(lib, bits):
    """Logits and every group's hidden values fit, whatever the tokens choose."""
    for rows, experts, top_k, shared in ((1, 256, 6, 1), (32, 512, 8, 8), (32, 3, 2, 0), (9, 8, 8, 1)):
        size = lib.moe_ffn_routed_workspace(ctypes.byref(_routed(bits, rows=rows, experts=experts, top_k=top_k, shared=shared)))
        assert size >= rows * experts * 4 + (min(rows * top_k, experts) + shared) * rows * 64 * 2
