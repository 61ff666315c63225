"""ctypes binding of libmoe_ffn.so (the C ABI in include/moe_ffn.h): argument marshalling only.

Every step of the block runs in the library's CUDA kernels.  There is no Python or CPU fallback: if
the library cannot be built or loaded, ``load()`` raises.
"""
from __future__ import annotations

import ctypes
import os
import re

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_ffn.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "moe_ffn.h")

c_i32, c_f32, c_vp = ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


class MoeFfnConfig(ctypes.Structure):
    _fields_ = [("hidden", c_i32), ("hc", c_i32), ("experts", c_i32), ("top_k", c_i32), ("inter", c_i32),
                ("shared_inter", c_i32), ("vocab", c_i32), ("n_layers", c_i32), ("hash_layer_count", c_i32),
                ("max_rows", c_i32), ("sinkhorn_iters", c_i32), ("rms_eps", c_f32)]


WEIGHT_FIELDS = ["hc_fn", "hc_base", "hc_scale", "ffn_norm", "gate", "exp_probs_b", "tid2eid", "gate_exps",
                 "up_exps", "down_exps", "gate_sh", "up_sh", "down_sh"]


class MoeFfnLayerWeights(ctypes.Structure):
    _fields_ = [(n, c_vp) for n in WEIGHT_FIELDS]


class MoeFfnHcWeights(ctypes.Structure):
    _fields_ = [("hc_fn", c_vp), ("hc_base", c_vp), ("hc_scale", c_vp), ("norm", c_vp)]


SUBLAYER_ATTN, SUBLAYER_FFN = 0, 1

MXFP8_FIELDS = ["gate_exps", "gate_exps_scale", "up_exps", "up_exps_scale", "down_exps", "down_exps_scale",
                "gate_sh", "gate_sh_scale", "up_sh", "up_sh_scale", "down_sh", "down_sh_scale"]


class MoeFfnMxfp8Experts(ctypes.Structure):
    _fields_ = [(n, c_vp) for n in MXFP8_FIELDS]

c_i64, c_sz = ctypes.c_int64, ctypes.c_size_t

TYPE_F32, TYPE_BF16, TYPE_F16 = 0, 1, 2
GATE_NONE, GATE_VECTOR, GATE_TOKEN = 0, 1, 2


class MoeFfnBlockNormArgs(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("hidden", c_i32), ("stream_type", c_i32), ("block_type", c_i32),
                ("gate_type", c_i32), ("gate_kind", c_i32), ("rows_per_gate", c_i32), ("residual_scale", c_f32),
                ("eps", c_f32), ("state", c_vp), ("ld_state", c_i64), ("f", c_vp), ("ld_f", c_i64), ("gate", c_vp),
                ("norm_f", c_vp), ("norm_next", c_vp), ("out", c_vp), ("ld_out", c_i64), ("y", c_vp), ("ld_y", c_i64)]


class MoeFfnBlockNormGrads(ctypes.Structure):
    _fields_ = [("d_out", c_vp), ("ld_d_out", c_i64), ("d_y", c_vp), ("ld_d_y", c_i64), ("d_state", c_vp),
                ("ld_d_state", c_i64), ("d_f", c_vp), ("ld_d_f", c_i64), ("d_gate", c_vp), ("d_norm_f", c_vp),
                ("d_norm_next", c_vp), ("workspace", c_vp), ("workspace_bytes", c_sz)]


ACTIVATIONS = {"silu": 0, "gelu": 1}


class MoeFfnGatedArgs(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("hidden", c_i32), ("inter", c_i32), ("type", c_i32), ("activation", c_i32),
                ("x", c_vp), ("ld_x", c_i64), ("w_gate", c_vp), ("w_up", c_vp), ("w_down", c_vp), ("y", c_vp),
                ("ld_y", c_i64), ("gate", c_vp), ("up", c_vp), ("d_y", c_vp), ("ld_d_y", c_i64), ("d_x", c_vp),
                ("ld_d_x", c_i64), ("d_w_gate", c_vp), ("d_w_up", c_vp), ("d_w_down", c_vp), ("workspace", c_vp),
                ("workspace_bytes", c_sz)]


TYPE_E4M3, TYPE_E5M2 = 0, 1
TILES_FORWARD, TILES_BACKWARD, TILES_BACKWARD_X, TILES_BACKWARD_WEIGHTS, TILES_FP8 = range(5)


class MoeFfnFp8MatmulArgs(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("n", c_i32), ("k", c_i32), ("a_type", c_i32), ("b_type", c_i32), ("out_type", c_i32),
                ("a", c_vp), ("ld_a", c_i64), ("a_scale", c_vp), ("b", c_vp), ("ld_b", c_i64), ("b_scale", c_vp),
                ("out", c_vp), ("ld_out", c_i64)]


class MoeFfnFp8QuantiseArgs(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("k", c_i32), ("type", c_i32), ("code_type", c_i32), ("block_rows", c_i32),
                ("pow2", c_i32), ("x", c_vp), ("ld_x", c_i64), ("codes", c_vp), ("ld_codes", c_i64), ("scales", c_vp)]


class MoeFfnFp8Out(ctypes.Structure):
    _fields_ = [("code_type", c_i32), ("pow2", c_i32), ("codes", c_vp), ("ld_codes", c_i64), ("scales", c_vp)]


class MoeFfnGatedQuantiseArgs(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("columns", c_i32), ("type", c_i32), ("activation", c_i32), ("gate", c_vp),
                ("ld_gate", c_i64), ("up", c_vp), ("ld_up", c_i64)]


class MoeFfnInt4WeightsArgs(ctypes.Structure):
    _fields_ = [("n", c_i32), ("k", c_i32), ("group", c_i32), ("scale_type", c_i32), ("codes", c_vp), ("scales", c_vp),
                ("zeros", c_vp)]


class MoeFfnInt4MatmulArgs(ctypes.Structure):
    _fields_ = [("rows", c_i32), ("n", c_i32), ("k", c_i32), ("type", c_i32), ("group", c_i32), ("x", c_vp),
                ("ld_x", c_i64), ("codes", c_vp), ("scales", c_vp), ("zeros", c_vp), ("out", c_vp), ("ld_out", c_i64),
                ("workspace", c_vp), ("workspace_bytes", c_sz)]


SCORES = {"sigmoid": 0, "softmax": 1}


class MoeFfnMatrices(ctypes.Structure):
    _fields_ = [("w", c_vp), ("scales", c_vp), ("zeros", c_vp)]


class MoeFfnRoutedArgs(ctypes.Structure):
    _fields_ = [(n, c_i32) for n in ("rows", "hidden", "inter", "experts", "top_k", "shared", "type", "router_type", "bits",
                                     "group", "score", "normalise", "activation")] + [
        ("route_scale", c_f32), ("x", c_vp), ("ld_x", c_i64), ("router", c_vp), ("bias", c_vp),
        *[(n, MoeFfnMatrices) for n in ("gate", "up", "down", "shared_gate", "shared_up", "shared_down")],
        ("y", c_vp), ("ld_y", c_i64), ("indices", c_vp), ("weights", c_vp), ("workspace", c_vp), ("workspace_bytes", c_sz)]


# return codes and device status bits (include/moe_ffn.h)
OK, ERR_NULL_PTR, ERR_BAD_CONFIG, ERR_LAYER_RANGE, ERR_ROWS_ZERO, ERR_ROWS_RANGE = 0, -1, -2, -3, -4, -5
ERR_NO_ROUTING_SOURCE, ERR_ALIAS, ERR_CUDA, ERR_NO_MEMORY, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_NO_WEIGHTS = (
    -6, -7, -8, -9, -10, -11, -12)
DEV_TOKEN_RANGE, DEV_ROUTE_RANGE, DEV_NONFINITE, DEV_TIMEOUT = 0x1, 0x2, 0x4, 0x8

_lib = None
build_error = None  # why load() could not build what was missing or out of date, where it went on without


def declared_functions() -> list[str]:
    """Names of the functions include/moe_ffn.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:int|int64_t|void|const char \*)\s*(moe_ffn_\w+)\s*\(", text, re.M)))


def load(build: bool = True):
    """Loads the library, building it first when it is missing or older than its sources."""
    global _lib, build_error
    if _lib is not None:
        return _lib
    if build:
        from . import build as _build
        try:
            _build.build()
            build_error = None
        except RuntimeError as e:
            build_error = e
            if not os.path.exists(LIB_PATH):
                raise
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m deepseek_v4_moe_gb300.build")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32 = c_vp, c_i32
    lib.moe_ffn_init.argtypes = [ctypes.POINTER(MoeFfnConfig), ctypes.POINTER(MoeFfnLayerWeights),
                                 ctypes.POINTER(vp)]
    lib.moe_ffn_init.restype = ctypes.c_int
    lib.moe_ffn_forward.argtypes = [vp, vp, vp, i32, i32, vp, vp]
    lib.moe_ffn_forward.restype = ctypes.c_int
    lib.moe_ffn_forward_layers.argtypes = [vp, vp, vp, i32, i32, i32, vp, vp]
    lib.moe_ffn_forward_layers.restype = ctypes.c_int
    lib.moe_ffn_forward_host.argtypes = [vp, vp, vp, i32, i32, vp, vp]
    lib.moe_ffn_forward_host.restype = ctypes.c_int
    lib.moe_ffn_status.argtypes = [vp]
    lib.moe_ffn_status.restype = ctypes.c_int
    lib.moe_ffn_debug_copy.argtypes = [vp, i32, vp, ctypes.c_size_t]
    lib.moe_ffn_debug_copy.restype = ctypes.c_int
    lib.moe_ffn_set_stage_timing.argtypes = [vp, i32]
    lib.moe_ffn_set_stage_timing.restype = ctypes.c_int
    lib.moe_ffn_stage_times.argtypes = [vp, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_char_p), i32]
    lib.moe_ffn_stage_times.restype = ctypes.c_int
    lib.moe_ffn_hc_split_noalloc.argtypes = [vp, vp, vp, vp, i32, i32, i32, i32, c_f32, vp, vp, vp, vp]
    lib.moe_ffn_hc_split_noalloc.restype = ctypes.c_int
    lib.moe_ffn_set_mxfp8_experts.argtypes = [vp, i32, ctypes.POINTER(MoeFfnMxfp8Experts)]
    lib.moe_ffn_set_mxfp8_experts.restype = ctypes.c_int
    lib.moe_ffn_set_attn_hc.argtypes = [vp, i32, ctypes.POINTER(MoeFfnHcWeights)]
    lib.moe_ffn_set_attn_hc.restype = ctypes.c_int
    lib.moe_ffn_hc_pre.argtypes = [vp, i32, i32, vp, i32, vp, vp, vp, vp, vp]
    lib.moe_ffn_hc_pre.restype = ctypes.c_int
    lib.moe_ffn_hc_post.argtypes = [vp, vp, vp, vp, vp, i32, vp, vp]
    lib.moe_ffn_hc_post.restype = ctypes.c_int
    lib.moe_ffn_set_fault_injection.argtypes = [vp, i32, ctypes.c_uint32]
    lib.moe_ffn_set_fault_injection.restype = ctypes.c_int
    norm, grads = ctypes.POINTER(MoeFfnBlockNormArgs), ctypes.POINTER(MoeFfnBlockNormGrads)
    lib.moe_ffn_block_norm.argtypes = [norm, vp]
    lib.moe_ffn_block_norm.restype = ctypes.c_int
    lib.moe_ffn_block_norm_workspace.argtypes = [norm, grads]
    lib.moe_ffn_block_norm_workspace.restype = c_i64
    lib.moe_ffn_block_norm_backward.argtypes = [norm, grads, vp]
    lib.moe_ffn_block_norm_backward.restype = ctypes.c_int
    gated = ctypes.POINTER(MoeFfnGatedArgs)
    lib.moe_ffn_gated_forward.argtypes = [gated, vp]
    lib.moe_ffn_gated_forward.restype = ctypes.c_int
    lib.moe_ffn_gated_backward.argtypes = [gated, vp]
    lib.moe_ffn_gated_backward.restype = ctypes.c_int
    lib.moe_ffn_gated_workspace.argtypes = [gated, i32]
    lib.moe_ffn_gated_workspace.restype = c_i64
    lib.moe_ffn_dense_status.argtypes = [vp]
    lib.moe_ffn_dense_status.restype = ctypes.c_int
    lib.moe_ffn_dense_fault_injection.argtypes = [i32, ctypes.c_uint32]
    lib.moe_ffn_dense_fault_injection.restype = ctypes.c_int
    lib.moe_ffn_dense_tiles.argtypes = [i32, i32, i32, i32, i32, ctypes.POINTER(i32)]
    lib.moe_ffn_dense_tiles.restype = ctypes.c_int
    lib.moe_ffn_fp8_matmul.argtypes = [ctypes.POINTER(MoeFfnFp8MatmulArgs), vp]
    lib.moe_ffn_fp8_matmul.restype = ctypes.c_int
    lib.moe_ffn_fp8_quantise.argtypes = [ctypes.POINTER(MoeFfnFp8QuantiseArgs), vp]
    lib.moe_ffn_fp8_quantise.restype = ctypes.c_int
    out8 = ctypes.POINTER(MoeFfnFp8Out)
    lib.moe_ffn_block_norm_fp8.argtypes = [norm, out8, vp]
    lib.moe_ffn_block_norm_fp8.restype = ctypes.c_int
    lib.moe_ffn_gated_quantise.argtypes = [ctypes.POINTER(MoeFfnGatedQuantiseArgs), out8, vp]
    lib.moe_ffn_gated_quantise.restype = ctypes.c_int
    int4 = ctypes.POINTER(MoeFfnInt4WeightsArgs)
    lib.moe_ffn_int4_quantise.argtypes = [int4, vp, i32, c_i64, vp]
    lib.moe_ffn_int4_quantise.restype = ctypes.c_int
    lib.moe_ffn_int4_widen.argtypes = [int4, vp, c_i64, vp]
    lib.moe_ffn_int4_widen.restype = ctypes.c_int
    lib.moe_ffn_int4_matmul.argtypes = [ctypes.POINTER(MoeFfnInt4MatmulArgs), vp]
    lib.moe_ffn_int4_matmul.restype = ctypes.c_int
    lib.moe_ffn_int4_matmul_workspace.argtypes = [ctypes.POINTER(MoeFfnInt4MatmulArgs)]
    lib.moe_ffn_int4_matmul_workspace.restype = c_i64
    lib.moe_ffn_routed_forward.argtypes = [ctypes.POINTER(MoeFfnRoutedArgs), vp]
    lib.moe_ffn_routed_forward.restype = ctypes.c_int
    lib.moe_ffn_routed_workspace.argtypes = [ctypes.POINTER(MoeFfnRoutedArgs)]
    lib.moe_ffn_routed_workspace.restype = c_i64
    lib.moe_ffn_last_error.argtypes = [vp]
    lib.moe_ffn_last_error.restype = ctypes.c_char_p
    lib.moe_ffn_destroy.argtypes = [vp]
    lib.moe_ffn_destroy.restype = None
    _lib = lib
    return lib
