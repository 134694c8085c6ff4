"""ctypes view of the C ABI in include/kda.h (libkda.so).

Only argument marshalling lives here.  If the library is missing this module
raises: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkda.so")

KDA_DTYPE_BF16 = 0
KDA_DTYPE_FP32 = 1
KDA_FLAG_QK_L2NORM = 1
KDA_FLAG_GATE_SOFTPLUS = 2
KDA_FLAG_SCALAR_GATE = 4
KDA_SCAN_DT_SOFTPLUS = 1
KDA_CONV_SILU = 1
KDA_ROTARY_INTERLEAVED = 1
KDA_ATTENTION_CAUSAL = 1

STATUS = {
    0: "KDA_OK", 1: "KDA_ERR_NULL_POINTER", 2: "KDA_ERR_BAD_SHAPE", 3: "KDA_ERR_UNSUPPORTED",
    4: "KDA_ERR_WORKSPACE_TOO_SMALL", 5: "KDA_ERR_BAD_STRUCT", 6: "KDA_ERR_HIP", 7: "KDA_ERR_ALIAS",
}
STATUS_CODE = {v: k for k, v in STATUS.items()}

# Every function declared in include/kda.h.
EXPORTS = ("kda_chunk_fwd_workspace_bytes", "kda_chunk_fwd", "kda_recurrent_fwd", "kda_recurrent_step",
           "kda_recurrent_bwd_workspace_bytes", "kda_recurrent_bwd", "kda_chunk_bwd_workspace_bytes",
           "kda_chunk_bwd", "kda_dplr_recurrent_fwd",
           "kda_status_string", "kda_last_error", "kda_last_hip_error", "kda_abi_version", "kda_version",
           "kda_chunk_fwd_noalloc", "kda_chunk_fwd_noalloc_max_workspace_bytes", "kda_dplr_chunk_fwd",
           "kda_dplr_chunk_fwd_workspace_bytes",
           "kda_selective_scan_fwd_workspace_bytes", "kda_selective_scan_fwd", "kda_selective_scan_step",
           "kda_selective_scan_bwd_workspace_bytes", "kda_selective_scan_bwd", "kda_short_conv_fwd",
           "kda_short_conv_step", "kda_short_conv_bwd_workspace_bytes", "kda_short_conv_bwd",
           "kda_layer_norm_fwd", "kda_layer_norm_bwd_workspace_bytes", "kda_layer_norm_bwd",
           "kda_rotary_fwd", "kda_rotary_bwd", "kda_latent_cache_append",
           "kda_latent_attention_step_workspace_bytes", "kda_latent_attention_step", "kda_latent_attention_fwd",
           "kda_latent_attention_bwd_workspace_bytes", "kda_latent_attention_bwd")

vp = ctypes.c_void_p


class ChunkFwdArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("q", vp), ("k", vp), ("v", vp), ("g", vp), ("beta", vp),
        ("initial_state", vp), ("final_state", vp), ("o", vp), ("cu_seqlens", vp),
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("chunk_size", ctypes.c_int32),
        ("workspace", vp), ("workspace_bytes", ctypes.c_size_t),
        ("stream", vp),
        ("flags", ctypes.c_uint32), ("gate_scale", ctypes.c_float),
    ]


class RecurrentStepArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("q", vp), ("k", vp), ("v", vp), ("g", vp), ("beta", vp),
        ("initial_state", vp), ("final_state", vp), ("o", vp),
        ("N", ctypes.c_int32), ("H", ctypes.c_int32), ("dk", ctypes.c_int32), ("dv", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("stream", vp),
        ("flags", ctypes.c_uint32), ("gate_scale", ctypes.c_float),
    ]


class RecurrentBwdArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("q", vp), ("k", vp), ("v", vp), ("g", vp), ("beta", vp),
        ("initial_state", vp), ("grad_o", vp), ("grad_final_state", vp),
        ("grad_q", vp), ("grad_k", vp), ("grad_v", vp), ("grad_g", vp), ("grad_beta", vp),
        ("grad_initial_state", vp), ("cu_seqlens", vp),
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("in_dtype", ctypes.c_int),
        ("workspace", vp), ("workspace_bytes", ctypes.c_size_t),
        ("stream", vp),
        ("flags", ctypes.c_uint32), ("gate_scale", ctypes.c_float),
    ]


class DplrArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("q", vp), ("k", vp), ("v", vp), ("g", vp), ("a", vp), ("b", vp),
        ("initial_state", vp), ("final_state", vp), ("o", vp), ("cu_seqlens", vp),
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("stream", vp),
    ]


class DplrChunkArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("q", vp), ("k", vp), ("v", vp), ("g", vp), ("a", vp), ("b", vp),
        ("initial_state", vp), ("final_state", vp), ("o", vp), ("cu_seqlens", vp),
        ("B", ctypes.c_int32), ("T", ctypes.c_int32), ("H", ctypes.c_int32),
        ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("in_dtype", ctypes.c_int), ("out_dtype", ctypes.c_int),
        ("workspace", vp), ("workspace_bytes", ctypes.c_size_t),
        ("stream", vp),
    ]


def _fields(spec: str):
    """Fields from "type: name name ..." lines: p pointer, l int64, i int32, f float, d dtype, u flags, z size."""
    kinds = dict(p=vp, l=ctypes.c_int64, i=ctypes.c_int32, f=ctypes.c_float, d=ctypes.c_int, u=ctypes.c_uint32,
                 z=ctypes.c_size_t)
    return [(name, kinds[line.split(":")[0].strip()]) for line in spec.strip().splitlines()
            for name in line.split(":")[1].split()]


class SelectiveScanArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: u dt A B C D z dt_bias initial_state final_state y cu_seqlens
        l: u_stride dt_stride B_stride C_stride z_stride y_stride
        i: batch T dim ds num_seqs
        d: in_dtype out_dtype
        p: workspace
        z: workspace_bytes
        p: stream
        u: flags""")


class SelectiveScanBwdArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: u dt A B C D z dt_bias initial_state grad_y grad_final_state
        p: grad_u grad_dt grad_A grad_B grad_C grad_D grad_z grad_dt_bias grad_initial_state cu_seqlens
        l: u_stride dt_stride B_stride C_stride z_stride grad_y_stride
        l: grad_u_stride grad_dt_stride grad_B_stride grad_C_stride grad_z_stride
        i: batch T dim ds num_seqs
        d: in_dtype grad_dtype
        p: workspace
        z: workspace_bytes
        p: stream
        u: flags""")


class ShortConvArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: x weight bias initial_state final_state y cu_seqlens
        l: x_stride y_stride
        i: batch T dim width num_seqs
        d: in_dtype out_dtype w_dtype
        p: stream
        u: flags""")


class ShortConvBwdArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: x weight bias initial_state grad_y grad_final_state grad_x grad_weight grad_bias grad_initial_state
        p: cu_seqlens
        l: x_stride grad_y_stride grad_x_stride
        i: batch T dim width num_seqs
        d: in_dtype grad_dtype w_dtype
        p: workspace
        z: workspace_bytes
        p: stream
        u: flags""")


class LayerNormArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: x residual weight bias y residual_out
        l: x_stride residual_stride y_stride residual_out_stride rows
        i: dim
        f: eps
        d: x_dtype res_dtype w_dtype out_dtype
        p: stream""")


class LayerNormBwdArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: x grad_y weight grad_residual grad_x grad_weight grad_bias
        l: x_stride grad_y_stride grad_residual_stride grad_x_stride rows
        i: dim
        f: eps
        d: x_dtype gy_dtype res_dtype w_dtype grad_dtype
        p: workspace
        z: workspace_bytes
        p: stream""")


class RotaryArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: x y positions inv_freq
        l: x_stride x_head_stride y_stride y_head_stride rows
        i: heads dim rot offset
        f: scale
        d: dtype
        p: stream
        u: flags""")


class LatentAppendArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: latent rope cache slots positions inv_freq
        l: latent_stride rope_stride rows
        i: num_blocks page dl dr
        f: scale
        d: dtype
        p: stream
        u: flags""")


class LatentStepArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: q_latent q_rope cache block_table lengths o lse
        l: q_latent_stride q_latent_head_stride q_rope_stride q_rope_head_stride o_stride o_head_stride
        l: block_table_stride
        i: N H dl dr page num_blocks max_blocks
        f: scale
        d: in_dtype out_dtype
        p: workspace
        z: workspace_bytes
        p: stream""")


class LatentAttentionArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: q k k_rope v o lse cu_seqlens_q cu_seqlens_k
        l: q_stride q_head_stride k_stride k_head_stride k_rope_stride v_stride v_head_stride o_stride o_head_stride
        i: batch Tq Tk H dn dr dv num_seqs
        f: scale
        d: in_dtype out_dtype
        p: stream
        u: flags""")


class LatentAttentionBwdArgs(ctypes.Structure):
    _fields_ = _fields("""
        u: struct_size
        p: q k k_rope v o lse grad_o grad_q grad_k grad_k_rope grad_v cu_seqlens_q cu_seqlens_k
        l: q_stride q_head_stride k_stride k_head_stride k_rope_stride v_stride v_head_stride o_stride o_head_stride
        l: grad_o_stride grad_o_head_stride grad_q_stride grad_q_head_stride grad_k_stride grad_k_head_stride
        l: grad_k_rope_stride grad_v_stride grad_v_head_stride
        i: batch Tq Tk H dn dr dv num_seqs
        f: scale
        d: in_dtype grad_dtype
        p: workspace
        z: workspace_bytes
        p: stream
        u: flags""")


# The layer operators' functions: their argument struct, and whether they return a size.
LAYER_FUNCTIONS = {
    "kda_selective_scan_fwd_workspace_bytes": (SelectiveScanArgs, True),
    "kda_selective_scan_fwd": (SelectiveScanArgs, False),
    "kda_selective_scan_step": (SelectiveScanArgs, False),
    "kda_selective_scan_bwd_workspace_bytes": (SelectiveScanBwdArgs, True),
    "kda_selective_scan_bwd": (SelectiveScanBwdArgs, False),
    "kda_short_conv_fwd": (ShortConvArgs, False),
    "kda_short_conv_step": (ShortConvArgs, False),
    "kda_short_conv_bwd_workspace_bytes": (ShortConvBwdArgs, True),
    "kda_short_conv_bwd": (ShortConvBwdArgs, False),
    "kda_layer_norm_fwd": (LayerNormArgs, False),
    "kda_layer_norm_bwd_workspace_bytes": (LayerNormBwdArgs, True),
    "kda_layer_norm_bwd": (LayerNormBwdArgs, False),
    "kda_rotary_fwd": (RotaryArgs, False),
    "kda_rotary_bwd": (RotaryArgs, False),
    "kda_latent_cache_append": (LatentAppendArgs, False),
    "kda_latent_attention_step_workspace_bytes": (LatentStepArgs, True),
    "kda_latent_attention_step": (LatentStepArgs, False),
    "kda_latent_attention_fwd": (LatentAttentionArgs, False),
    "kda_latent_attention_bwd_workspace_bytes": (LatentAttentionBwdArgs, True),
    "kda_latent_attention_bwd": (LatentAttentionBwdArgs, False),
}


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.name = STATUS.get(status, f"status {status}")
        super().__init__(f"{self.name}: {message}")


_lib = None


def load():
    """Load libkda.so (built by gated_delta_rule_52_amd.build); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m gated_delta_rule_52_amd.build` (there is no fallback)")
        lib = ctypes.CDLL(LIB_PATH)
        lib.kda_chunk_fwd_workspace_bytes.restype = ctypes.c_size_t
        lib.kda_chunk_fwd_workspace_bytes.argtypes = [ctypes.POINTER(ChunkFwdArgs)]
        lib.kda_chunk_fwd.restype = ctypes.c_int
        lib.kda_chunk_fwd.argtypes = [ctypes.POINTER(ChunkFwdArgs)]
        lib.kda_recurrent_fwd.restype = ctypes.c_int
        lib.kda_recurrent_fwd.argtypes = [ctypes.POINTER(ChunkFwdArgs)]
        lib.kda_recurrent_step.restype = ctypes.c_int
        lib.kda_recurrent_step.argtypes = [ctypes.POINTER(RecurrentStepArgs)]
        lib.kda_recurrent_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.kda_recurrent_bwd_workspace_bytes.argtypes = [ctypes.POINTER(RecurrentBwdArgs)]
        lib.kda_recurrent_bwd.restype = ctypes.c_int
        lib.kda_recurrent_bwd.argtypes = [ctypes.POINTER(RecurrentBwdArgs)]
        lib.kda_chunk_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.kda_chunk_bwd_workspace_bytes.argtypes = [ctypes.POINTER(RecurrentBwdArgs)]
        lib.kda_chunk_bwd.restype = ctypes.c_int
        lib.kda_chunk_bwd.argtypes = [ctypes.POINTER(RecurrentBwdArgs)]
        lib.kda_dplr_recurrent_fwd.restype = ctypes.c_int
        lib.kda_dplr_recurrent_fwd.argtypes = [ctypes.POINTER(DplrArgs)]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_status_string.argtypes = [ctypes.c_int]
        lib.kda_last_error.restype = ctypes.c_char_p
        lib.kda_last_error.argtypes = []
        lib.kda_last_hip_error.restype = ctypes.c_char_p
        lib.kda_last_hip_error.argtypes = []
        lib.kda_abi_version.restype = ctypes.c_int
        lib.kda_abi_version.argtypes = []
        lib.kda_version.restype = ctypes.c_int
        lib.kda_version.argtypes = []
        lib.kda_chunk_fwd_noalloc.restype = ctypes.c_int
        lib.kda_chunk_fwd_noalloc.argtypes = [ctypes.POINTER(ChunkFwdArgs)]
        lib.kda_chunk_fwd_noalloc_max_workspace_bytes.restype = ctypes.c_size_t
        lib.kda_chunk_fwd_noalloc_max_workspace_bytes.argtypes = []
        lib.kda_dplr_chunk_fwd.restype = ctypes.c_int
        lib.kda_dplr_chunk_fwd.argtypes = [ctypes.POINTER(DplrChunkArgs)]
        lib.kda_dplr_chunk_fwd_workspace_bytes.restype = ctypes.c_size_t
        lib.kda_dplr_chunk_fwd_workspace_bytes.argtypes = [ctypes.POINTER(DplrChunkArgs)]
        for name, (args_struct, size) in LAYER_FUNCTIONS.items():
            fn = getattr(lib, name)
            fn.argtypes = [ctypes.POINTER(args_struct)]
            fn.restype = ctypes.c_size_t if size else ctypes.c_int
        _lib = lib
    return _lib


def check(status: int):
    if status != 0:
        raise KdaError(status, load().kda_last_error().decode())


def chunk_fwd_raw(args: ChunkFwdArgs) -> int:
    args.struct_size = ctypes.sizeof(ChunkFwdArgs)
    return load().kda_chunk_fwd(ctypes.byref(args))


def dplr_chunk_fwd_raw(args: DplrChunkArgs) -> int:
    args.struct_size = ctypes.sizeof(DplrChunkArgs)
    return load().kda_dplr_chunk_fwd(ctypes.byref(args))


def dplr_chunk_workspace_raw(args: DplrChunkArgs) -> int:
    args.struct_size = ctypes.sizeof(DplrChunkArgs)
    return load().kda_dplr_chunk_fwd_workspace_bytes(ctypes.byref(args))


def chunk_fwd_noalloc_raw(args: ChunkFwdArgs) -> int:
    args.struct_size = ctypes.sizeof(ChunkFwdArgs)
    return load().kda_chunk_fwd_noalloc(ctypes.byref(args))


def chunk_workspace_raw(args: ChunkFwdArgs) -> int:
    args.struct_size = ctypes.sizeof(ChunkFwdArgs)
    return load().kda_chunk_fwd_workspace_bytes(ctypes.byref(args))


def recurrent_fwd_raw(args: ChunkFwdArgs) -> int:
    args.struct_size = ctypes.sizeof(ChunkFwdArgs)
    return load().kda_recurrent_fwd(ctypes.byref(args))


def recurrent_step_raw(args: RecurrentStepArgs) -> int:
    args.struct_size = ctypes.sizeof(RecurrentStepArgs)
    return load().kda_recurrent_step(ctypes.byref(args))


def recurrent_bwd_raw(args: RecurrentBwdArgs) -> int:
    args.struct_size = ctypes.sizeof(RecurrentBwdArgs)
    return load().kda_recurrent_bwd(ctypes.byref(args))


def recurrent_bwd_workspace_raw(args: RecurrentBwdArgs) -> int:
    args.struct_size = ctypes.sizeof(RecurrentBwdArgs)
    return load().kda_recurrent_bwd_workspace_bytes(ctypes.byref(args))


def chunk_bwd_raw(args: RecurrentBwdArgs) -> int:
    args.struct_size = ctypes.sizeof(RecurrentBwdArgs)
    return load().kda_chunk_bwd(ctypes.byref(args))


def chunk_bwd_workspace_raw(args: RecurrentBwdArgs) -> int:
    args.struct_size = ctypes.sizeof(RecurrentBwdArgs)
    return load().kda_chunk_bwd_workspace_bytes(ctypes.byref(args))


def dplr_fwd_raw(args: DplrArgs) -> int:
    args.struct_size = ctypes.sizeof(DplrArgs)
    return load().kda_dplr_recurrent_fwd(ctypes.byref(args))


def layer_raw(name: str, args) -> int:
    """Calls one of LAYER_FUNCTIONS; args.struct_size is set here."""
    args.struct_size = ctypes.sizeof(args)
    return getattr(load(), name)(ctypes.byref(args))


_CODES = {vp: "P", ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_int: "i", ctypes.c_float: "f",
          ctypes.c_uint32: "I", ctypes.c_size_t: "N"}


def packer(args_struct) -> struct.Struct:
    """The layout of an argument struct as struct.Struct: packing one by position takes a third of the time that a
    ctypes object does.  Pointers are integers there, 0 for NULL."""
    return struct.Struct("@" + "".join(_CODES[kind] for _, kind in args_struct._fields_) + "0P")


_layer_functions = {}


def layer_function(name: str):
    """The loaded library's function of this name, taking a packed argument struct."""
    fn = _layer_functions.get(name)
    if fn is None:
        fn = load()[name]  # a function object of its own
        fn.argtypes = [ctypes.c_char_p]
        fn.restype = ctypes.c_size_t if LAYER_FUNCTIONS[name][1] else ctypes.c_int
        _layer_functions[name] = fn
    return fn
