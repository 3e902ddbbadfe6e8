"""ctypes loader for ``libkda.so`` (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os
import struct

LIBRARY = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkda.so")

# Every symbol include/kda.h declares.
EXPORTS = ("kda_fwd", "kda_fwd_ex", "kda_fwd_scan", "kda_fwd_scan_static",
           "kda_fwd_scan_workspace_bytes", "kda_status_string", "kda_fwd_kernel",
           "kda_abi_version", "kda_short_conv", "kda_ssm_fwd", "kda_ssm_workspace_bytes",
           "kda_gated_norm", "kda_residual_norm", "kda_delta_fwd", "kda_delta_workspace_bytes",
           "kda_qk_norm_rotary", "kda_append_kv", "kda_paged_attention", "kda_paged_attention_workspace_bytes")
SCAN_STATIC_BYTES = 32 << 20  # KDA_SCAN_STATIC_BYTES
ABI_VERSION = 6

# kda_status codes (include/kda.h)
KDA_OK = 0
KDA_ERR_NULL_POINTER = 1
KDA_ERR_HEAD_DIM = 2
KDA_ERR_LOWER_BOUND = 3
KDA_ERR_VARLEN_BATCH = 4
KDA_ERR_STATE_DTYPE = 5
KDA_ERR_ALIAS = 6
KDA_ERR_SIZE = 7
KDA_ERR_SCALE = 8
KDA_ERR_LAUNCH = 9
KDA_ERR_WORKSPACE = 10
KDA_ERR_ALIGNMENT = 11
KDA_ERR_OPTION = 12
KDA_ERR_SHAPE = 13
KDA_ERR_DTYPE = 14
KDA_ERR_STRIDE = 15

# kda_dtype codes
KDA_DTYPE_NONE = 0
KDA_DTYPE_BF16 = 1
KDA_DTYPE_FP32 = 2

# kda_options fields
KDA_KERNEL_AUTO, KDA_KERNEL_CHUNKED, KDA_KERNEL_RECURRENT, KDA_KERNEL_SINGLE = 0, 1, 2, 3
KDA_INVERSE_SUBSTITUTION, KDA_INVERSE_NEUMANN = 0, 1
KDA_SIGMOID_EXP2, KDA_SIGMOID_TANH = 0, 1

# kda_activation codes
KDA_ACT_NONE, KDA_ACT_SILU, KDA_ACT_SIGMOID = 0, 1, 2


class Options(ctypes.Structure):
    """struct kda_options"""
    _fields_ = [("kernel", ctypes.c_int32), ("inverse", ctypes.c_int32),
                ("sigmoid", ctypes.c_int32), ("reserved", ctypes.c_int32)]


_P, _I64, _I32, _F64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double


def _fields(kind, names):
    return [(n, kind) for n in names.split()]


class ConvArgs(ctypes.Structure):
    """struct kda_conv_args"""
    _fields_ = (_fields(_P, "x") + _fields(_I64, "x_stride_b x_stride_t")
                + _fields(_P, "weight bias out initial_state final_state cu_seqlens")
                + _fields(_I64, "num_seqs B T D W")
                + _fields(_I32, "weight_dtype initial_state_dtype final_state_dtype activation")
                + _fields(_I64, "l2norm") + _fields(_F64, "l2norm_eps") + _fields(_I64, "reserved"))


class SsmArgs(ctypes.Structure):
    """struct kda_ssm_args"""
    _fields_ = (_fields(_P, "x dt b c z out")
                + _fields(_I64, "x_stride_b x_stride_t dt_stride_b dt_stride_t b_stride_b b_stride_t "
                                "c_stride_b c_stride_t z_stride_b z_stride_t")
                + _fields(_P, "A_log D dt_bias initial_state final_state cu_seqlens")
                + _fields(_I64, "num_seqs B T H P G N")
                + _fields(_I32, "initial_state_dtype final_state_dtype softplus reserved")
                + _fields(_I64, "seg_tokens") + _fields(_P, "workspace") + _fields(_I64, "workspace_bytes"))


class GatedNormArgs(ctypes.Structure):
    """struct kda_gated_norm_args"""
    _fields_ = (_fields(_P, "x gate weight out") + _fields(_I64, "x_stride gate_stride rows D group")
                + _fields(_I32, "weight_dtype activation gate_first reserved") + _fields(_F64, "eps"))


class ResidualNormArgs(ctypes.Structure):
    """struct kda_residual_norm_args"""
    _fields_ = (_fields(_P, "x residual residual_out post_weight gate weight out")
                + _fields(_I64, "x_stride gate_stride gate_period rows D")
                + _fields(_I32, "residual_dtype residual_out_dtype post_weight_dtype gate_dtype weight_dtype "
                                "reserved")
                + _fields(_F64, "residual_scale block_scale eps"))


class DeltaArgs(ctypes.Structure):
    """struct kda_delta_args"""
    _fields_ = (_fields(_P, "q k v g beta out")
                + _fields(_I64, "q_stride_b q_stride_t k_stride_b k_stride_t v_stride_b v_stride_t "
                                "g_stride_b g_stride_t beta_stride_b beta_stride_t")
                + _fields(_P, "A_log dt_bias initial_state final_state cu_seqlens")
                + _fields(_I64, "num_seqs B T H G K V")
                + _fields(_I32, "initial_state_dtype final_state_dtype") + _fields(_I64, "reserved")
                + _fields(_F64, "scale") + _fields(_I64, "seg_tokens") + _fields(_P, "workspace")
                + _fields(_I64, "workspace_bytes"))


class RotaryArgs(ctypes.Structure):
    """struct kda_rotary_args"""
    _fields_ = (_fields(_P, "q k q_out k_out") + _fields(_I64, "q_stride_b q_stride_t k_stride_b k_stride_t")
                + _fields(_P, "positions inv_freq q_weight k_weight") + _fields(_I64, "B T Hq Hk D R")
                + _fields(_I32, "q_weight_dtype k_weight_dtype interleaved reserved")
                + _fields(_F64, "eps rotary_scale"))


class AppendArgs(ctypes.Structure):
    """struct kda_append_args"""
    _fields_ = (_fields(_P, "k v k_cache v_cache") + _fields(_I64, "k_stride_b k_stride_t v_stride_b v_stride_t "
                "k_cache_stride_page k_cache_stride_token k_cache_stride_head "
                "v_cache_stride_page v_cache_stride_token v_cache_stride_head")
                + _fields(_P, "slots positions inv_freq weight") + _fields(_I64, "B T Hk D R pages page_size")
                + _fields(_I32, "weight_dtype interleaved") + _fields(_I64, "reserved")
                + _fields(_F64, "eps rotary_scale"))


class AttentionArgs(ctypes.Structure):
    """struct kda_attention_args"""
    _fields_ = (_fields(_P, "q k_cache v_cache block_table lengths out lse")
                + _fields(_I64, "q_stride table_stride k_cache_stride_page k_cache_stride_token k_cache_stride_head "
                                "v_cache_stride_page v_cache_stride_token v_cache_stride_head "
                                "N Hq Hk D pages page_size table_width window reserved")
                + _fields(_F64, "scale") + _fields(_P, "workspace") + _fields(_I64, "workspace_bytes"))


class KdaLibraryMissing(RuntimeError):
    """libkda.so has not been built (there is no other implementation)."""


_lib = None


def packer(args):
    """A function that packs the fields of a ctypes Structure into bytes (a fifth of the time the Structure takes)."""
    packed = struct.Struct("@" + "".join({_P: "P", _I64: "q", _I32: "i", _F64: "d"}[kind] for _, kind in args._fields_))
    assert packed.size == ctypes.sizeof(args)
    return packed.pack


# The layer operators' entry points, taking the bytes of their arguments, and what packs those; filled by load().
LAYER = {}


def load() -> ctypes.CDLL:
    """Load libkda.so once and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY):
        raise KdaLibraryMissing(
            f"{LIBRARY} is missing; build it with `python -m gated_delta_rule_36_amd.build`")
    lib = ctypes.CDLL(LIBRARY)
    lib.kda_abi_version.argtypes = []
    lib.kda_abi_version.restype = ctypes.c_int
    if lib.kda_abi_version() != ABI_VERSION:
        raise KdaLibraryMissing(f"{LIBRARY} has ABI {lib.kda_abi_version()}, expected {ABI_VERSION}")
    p, i64, d = ctypes.c_void_p, ctypes.c_int64, ctypes.c_double
    lib.kda_fwd.argtypes = [p, p, p, p, p, d, p, p, p, d, p, ctypes.c_int, p, ctypes.c_int,
                            p, i64, i64, i64, i64, i64, i64, p]
    lib.kda_fwd.restype = ctypes.c_int
    opt = ctypes.POINTER(Options)
    lib.kda_fwd_ex.argtypes = [p, p, p, p, p, d, p, p, p, d, p, ctypes.c_int, p, ctypes.c_int,
                               p, i64, i64, i64, i64, i64, i64, opt, p]
    lib.kda_fwd_ex.restype = ctypes.c_int
    lib.kda_fwd_scan.argtypes = [p, p, p, p, p, d, p, p, p, d, p, ctypes.c_int, p, ctypes.c_int,
                                 p, i64, i64, i64, i64, i64, i64, i64, p, i64, opt, p]
    lib.kda_fwd_scan.restype = ctypes.c_int
    lib.kda_fwd_scan_static.argtypes = [p, p, p, p, p, d, p, p, p, d, p, ctypes.c_int, p,
                                        ctypes.c_int, p, i64, i64, i64, i64, i64, i64, i64, opt, p]
    lib.kda_fwd_scan_static.restype = ctypes.c_int
    lib.kda_fwd_scan_workspace_bytes.argtypes = [p, i64, i64, i64, i64, i64]
    lib.kda_fwd_scan_workspace_bytes.restype = i64
    lib.kda_status_string.argtypes = [ctypes.c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_fwd_kernel.argtypes = [i64, ctypes.c_int, opt]
    lib.kda_fwd_kernel.restype = ctypes.c_char_p
    for name, args in (("kda_short_conv", ConvArgs), ("kda_ssm_fwd", SsmArgs),
                       ("kda_gated_norm", GatedNormArgs), ("kda_residual_norm", ResidualNormArgs),
                       ("kda_delta_fwd", DeltaArgs), ("kda_qk_norm_rotary", RotaryArgs),
                       ("kda_append_kv", AppendArgs), ("kda_paged_attention", AttentionArgs)):
        getattr(lib, name).argtypes = [ctypes.POINTER(args), p]
        getattr(lib, name).restype = ctypes.c_int
        LAYER[name] = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, p)((name, lib)), packer(args)
    for name, args in (("kda_ssm_workspace_bytes", SsmArgs), ("kda_delta_workspace_bytes", DeltaArgs),
                       ("kda_paged_attention_workspace_bytes", AttentionArgs)):
        getattr(lib, name).argtypes = [ctypes.POINTER(args)]
        getattr(lib, name).restype = i64
        LAYER[name] = ctypes.CFUNCTYPE(i64, ctypes.c_char_p)((name, lib)), packer(args)
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().kda_status_string(code).decode()
