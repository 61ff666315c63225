"""Row strides of block_norm so large that a row's place in memory would not be a 64-bit number are refused, as are
overlaps that such strides once hid; large ones that memory can have are not.  No GPU: the checks answer first."""
import ctypes

import pytest

import test_dense_abi as abi
from deepseek_v4_moe_gb300 import _lib

A = abi.A
ROWS = 1 << 30
NORM = ["ld_state", "ld_f", "ld_out", "ld_y"]
GRADS = ["ld_d_out", "ld_d_y", "ld_d_state", "ld_d_f"]


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def forward(lib, **kw):
    return lib.moe_ffn_block_norm(ctypes.byref(abi._norm(**kw)), None)


def backward(lib, kw, gkw):
    a, g = ctypes.byref(abi._norm(**kw)), ctypes.byref(abi._grads(**gkw))
    return lib.moe_ffn_block_norm_backward(a, g, None), lib.moe_ffn_block_norm_workspace(a, g)


@pytest.mark.parametrize("ld", [1 << 31, 1 << 34, (1 << 35) + 256, 1 << 62, (1 << 63) - 1])
@pytest.mark.parametrize("name", NORM)
def test_block_norm_refuses_strides_past_64_bits(lib, name, ld):
    assert forward(lib, rows=ROWS, **{name: ld}) == _lib.ERR_BAD_CONFIG, lib.moe_ffn_last_error(None)


@pytest.mark.parametrize("ld", [1 << 31, 1 << 34, (1 << 35) + 256, 1 << 62, (1 << 63) - 1])
@pytest.mark.parametrize("name", ["ld_state", "ld_f"] + GRADS)
def test_block_norm_backward_refuses_strides_past_64_bits(lib, name, ld):
    kw = {name: ld} if name in NORM else {}
    gkw = {name: ld} if name in GRADS else {}
    assert backward(lib, dict(rows=ROWS, **kw), gkw) == (_lib.ERR_BAD_CONFIG,) * 2, lib.moe_ffn_last_error(None)


def test_two_rows_as_far_apart_as_memory_is_long(lib):
    # the overlap is seen at a stride of 2^40 elements, and a tensor beside is not refused
    assert forward(lib, rows=2, ld_state=1 << 40, out=A + 512) == _lib.ERR_ALIAS
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not memory")
    far = {name: 1 << 40 for name in NORM}
    at = dict(state=A, f=A + 4096, out=A + 8192, y=A + 12288)
    assert forward(lib, rows=2, block_type=_lib.TYPE_F32, norm_f=None, norm_next=1 << 50, **far, **at) in (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED)


def test_one_row_has_any_stride(lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on addresses that are not memory")
    assert forward(lib, rows=1, ld_state=1 << 55, ld_out=1 << 55) in (_lib.ERR_CUDA, _lib.ERR_UNSUPPORTED)
