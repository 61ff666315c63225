"""Every instance of the dense sublayer's tensor-core kernels is run by the GPU tests: which tiles their sizes take is
asked of the code that chooses them, so a changed figure of its model that leaves an instance untested fails here.
(The list TILES of test_gpu_dense_edges.py alone leaves three out; MORE_TILES has them.)"""
import ctypes
import os
import re

import pytest

import test_gpu_dense_edges as edges
from deepseek_v4_moe_gb300 import _lib, build

SMS = 152
GRADIENTS = (_lib.TILES_BACKWARD, _lib.TILES_BACKWARD_X, _lib.TILES_BACKWARD_WEIGHTS)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def tiles(lib, call, rows, n, k, sms=SMS):
    out = (ctypes.c_int32 * 9)()
    count = lib.moe_ffn_dense_tiles(call, rows, n, k, sms, out)
    assert 0 <= count <= 3, lib.moe_ffn_last_error(None)
    return [tuple(out[3 * i:3 * i + 3]) for i in range(count)]


def instances(source):
    """What the launch functions instantiate, read from their macros: (product, columns, kind)."""
    text = open(os.path.join(build.CSRC, source)).read()
    kinds = {"kOneTile": 0, "kPairTile": 1, "kSplitTile": 2}
    products = {"kGateUp": 0, "kDown": 1, "kHiddenGrad": 2, "kGrads": 3}
    if "fp8" in source:
        return {(4, int(bn), kinds[k]) for bn, k in re.findall(r"^  MOE_LAUNCH\((\d+), (k\w+)\);", text, re.M)}
    every = {(int(bn), kinds[k]) for bn, k in re.findall(r"MOE_LAUNCH\(MODE, (\d+), (k\w+)\)", text)}
    found = {(products[p], *t) for p in re.findall(r"^  MOE_LAUNCH_ALL\((k\w+)\);", text, re.M) for t in every}
    return found | {(products[p], int(bn), kinds[k])
                    for p, bn, k in re.findall(r"^  MOE_LAUNCH\((k\w+), (\d+), (k\w+)\);", text, re.M)}


def test_every_instance_of_the_gated_block_is_run(lib):
    want = instances("dense_gemm.cu")
    assert len(want) == 34
    ran = set()
    for rows, hidden, inter in edges.TILES:
        for call in (_lib.TILES_FORWARD, _lib.TILES_BACKWARD):
            ran.update(tiles(lib, call, rows, inter, hidden))
    for rows, hidden, inter in edges.MORE_TILES:
        for call in (_lib.TILES_FORWARD, *GRADIENTS):
            ran.update(tiles(lib, call, rows, inter, hidden))
    assert ran == want, (sorted(want - ran), sorted(ran - want))


def test_every_instance_of_the_fp8_product_is_run(lib):
    want = instances("dense_fp8.cu")
    assert len(want) == 7
    ran = {t for rows, n, k in edges.TILES8 for t in tiles(lib, _lib.TILES_FP8, rows, n, k)}
    assert ran == want, (sorted(want - ran), sorted(ran - want))


def test_gradients_in_one_launch_and_in_two_are_run(lib):
    counts = {len(tiles(lib, _lib.TILES_BACKWARD, r, i, h)) for r, h, i in edges.MORE_TILES}
    assert counts == {2, 3}


@pytest.mark.parametrize("sms", [8, 76, 148, 152, 160])
def test_tiles_exist_on_any_number_of_sms(lib, sms):
    want, want8 = instances("dense_gemm.cu"), instances("dense_fp8.cu")
    for rows, hidden, inter in edges.TILES + edges.MORE_TILES:
        for call in (_lib.TILES_FORWARD, *GRADIENTS):
            assert set(tiles(lib, call, rows, inter, hidden, sms)) <= want
    for rows, n, k in edges.TILES8:
        assert set(tiles(lib, _lib.TILES_FP8, rows, n, k, sms)) <= want8


def test_few_rows_take_no_tile(lib):
    assert tiles(lib, _lib.TILES_FORWARD, 4, 2048, 4096) == [] == tiles(lib, _lib.TILES_FP8, 1, 4096, 4096)
    assert len(tiles(lib, _lib.TILES_FORWARD, 9, 2048, 4096)) == 2 and len(tiles(lib, _lib.TILES_FP8, 5, 64, 64)) == 1


@pytest.mark.parametrize("args,code", [
    ((9, 8, 64, 64, SMS), _lib.ERR_BAD_CONFIG), ((0, 8, 64, 64, 0), _lib.ERR_BAD_CONFIG),
    ((0, 0, 64, 64, SMS), _lib.ERR_ROWS_ZERO), ((1, 8, 60, 64, SMS), _lib.ERR_BAD_CONFIG),
    ((4, 0, 64, 64, SMS), _lib.ERR_BAD_CONFIG), ((4, 8, 64, 40, SMS), _lib.ERR_BAD_CONFIG),
    ((4, 8, 0, 64, SMS), _lib.ERR_BAD_CONFIG), ((4, 8, 64, (1 << 20) + 16, SMS), _lib.ERR_BAD_CONFIG)])
def test_tiles_refuses(lib, args, code):
    assert lib.moe_ffn_dense_tiles(*args, (ctypes.c_int32 * 9)()) == code
    assert lib.moe_ffn_dense_tiles(0, 8, 64, 64, SMS, None) == _lib.ERR_NULL_PTR
