"""Deterministic, batch-invariant joint attention of a Qwen-Image MMDiT block
(forward and backward, with the QK-RMSNorm + three-axis RoPE prologue) for one
NVIDIA GB300.

This module is a thin binding over the C ABI of ``librlk_joint_attn.so``
(declared in ``include/rlk_joint_attn.h``): it marshals arguments and checks
shapes so that no bad pointer reaches the library. Every step of the path runs
in the library's CUDA kernels; there is no CPU or PyTorch fallback. If the
library is missing, loading it raises.

PyTorch is used only for device memory and streams.
"""

from __future__ import annotations

import ctypes
import operator
import os
from typing import Sequence

__all__ = [
    "Shape", "RlkError", "lib", "library_path", "load_library",
    "rlk_joint_attn_ctx_bytes", "rlk_joint_attn_bwd_workspace_bytes", "rlk_joint_attn_bwd_workspace_min_bytes",
    "rlk_joint_attn_fwd", "rlk_joint_attn_bwd", "rlk_joint_attn_check_status",
    "rlk_strict_math_compiled", "rlk_joint_attn_trace", "rlk_strerror",
    "rlk_kernel_timing", "rlk_kernel_timing_read", "rlk_joint_attn_fwd_noalloc",
    "rlk_joint_attn_unfused_bytes", "rlk_qk_norm_rope", "rlk_joint_attn_qk_gemm",
    "rlk_joint_attn_softmax", "rlk_joint_attn_av_gemm", "UNFUSED", "JointAttention",
    "rlk_op_trace_enable", "rlk_op_trace_count", "rlk_op_trace_read", "op_trace", "OP_TRACE_CAP",
    "rlk_joint_attn_state_bytes", "rlk_joint_attn_fwd_shard", "rlk_joint_attn_fwd_streams",
    "rlk_joint_attn_bwd_streams", "rlk_qkv_bias_gemm", "rlk_joint_attn_fwd_ctx",
    "rlk_attn_out_bias_gemm", "rlk_selftest_wait_timeout", "rlk_fwd_tile_schedule", "FWD_TILES",
    "rlk_joint_attn_bwd_stats", "rlk_joint_attn_softmax_bwd", "rlk_joint_attn_av_gemm_bwd",
    "rlk_joint_attn_qk_gemm_bwd", "rlk_qk_norm_rope_bwd",
    "AdalnShape", "AdalnIo", "AdalnGrad", "rlk_adaln_workspace_bytes", "rlk_adaln_modulation_fwd",
    "rlk_adaln_modulation_bwd", "rlk_adaln_gate_residual_fwd", "rlk_adaln_gate_residual_bwd", "AdaLN", "NORMS",
    "AdamwTensor", "AdamwArgs", "rlk_adamw_step", "rlk_grad_norm", "rlk_grad_norm_workspace_bytes", "AdamW",
    "Fp8Quant", "Fp8Product", "rlk_fp8_row_bytes", "rlk_fp8_scale_row_bytes", "rlk_fp8_quant_workspace_bytes",
    "rlk_fp8_quantize", "rlk_fp8_gemm", "FP8_FORMATS", "FP8_MAX_ITEMS", "Fp8Projection",
    "MuonMatrix", "MuonArgs", "rlk_muon_workspace_bytes", "rlk_muon_step", "rlk_orthogonalize", "Muon", "orthogonalize",
    "EXPORTED_SYMBOLS", "KERNEL_IDS",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_NAME = "librlk_joint_attn.so"
HEAD_DIM = 128
AXES = (16, 56, 56)
MAX_BATCH = 256

RLK_OK = 0
STATUS_NAMES = {
    0: "RLK_OK", 1: "RLK_ERR_INVALID_ARG", 2: "RLK_ERR_UNSUPPORTED", 3: "RLK_ERR_ALIGNMENT",
    4: "RLK_ERR_WORKSPACE", 5: "RLK_ERR_CUDA", 6: "RLK_ERR_DEVICE_TIMEOUT",
}
KERNEL_IDS = {
    "rope_table": 0, "prologue": 1, "attn_fwd": 2, "bwd_pre": 3,
    "bwd_dkdv": 4, "bwd_dq": 5, "norm_rope_bwd_k": 6, "dg_fold": 7,
    "qk_gemm": 8, "softmax": 9, "av_gemm": 10, "attn_fwd_shard": 11, "qkv_gemm": 12, "out_gemm": 13,
    "dp_gemm": 14, "softmax_bwd": 15, "key_gemm": 16, "query_gemm": 17, "norm_rope_bwd_q": 18,
    "adaln_fwd": 19, "adaln_bwd": 20, "adaln_fold": 21, "grad_norm": 22, "grad_norm_fold": 23, "adamw": 24,
    "adaln_weight": 25, "fp8_quant": 26, "fp8_fold": 27, "fp8_gemm": 28, "muon_momentum": 29, "muon_start": 30,
    "muon_gram": 31, "muon_poly": 32, "muon_apply": 33, "muon_update": 34, "muon_small": 35,
}
# which intermediate rlk_joint_attn_unfused_bytes() sizes
UNFUSED = {"scores": 0, "p": 1, "alpha": 2, "rows": 3, "dp": 4, "ds": 5, "stats": 6, "dhat": 7, "gain_tiles": 8}
# Every symbol include/rlk_joint_attn.h declares.
EXPORTED_SYMBOLS = (
    "rlk_joint_attn_ctx_bytes", "rlk_joint_attn_bwd_workspace_bytes", "rlk_joint_attn_bwd_workspace_min_bytes",
    "rlk_joint_attn_fwd", "rlk_joint_attn_bwd", "rlk_joint_attn_check_status",
    "rlk_strict_math_compiled", "rlk_joint_attn_trace", "rlk_strerror",
    "rlk_kernel_timing", "rlk_kernel_timing_read", "rlk_joint_attn_fwd_noalloc",
    "rlk_joint_attn_unfused_bytes", "rlk_qk_norm_rope", "rlk_joint_attn_qk_gemm",
    "rlk_joint_attn_softmax", "rlk_joint_attn_av_gemm",
    "rlk_op_trace_enable", "rlk_op_trace_count", "rlk_op_trace_read",
    "rlk_joint_attn_state_bytes", "rlk_joint_attn_fwd_shard",
    "rlk_joint_attn_fwd_streams", "rlk_joint_attn_bwd_streams", "rlk_qkv_bias_gemm",
    "rlk_joint_attn_fwd_ctx", "rlk_attn_out_bias_gemm", "rlk_selftest_wait_timeout",
    "rlk_fwd_tile_schedule",
    "rlk_joint_attn_bwd_stats", "rlk_joint_attn_softmax_bwd", "rlk_joint_attn_av_gemm_bwd",
    "rlk_joint_attn_qk_gemm_bwd", "rlk_qk_norm_rope_bwd",
    "rlk_adaln_workspace_bytes", "rlk_adaln_modulation_fwd", "rlk_adaln_modulation_bwd",
    "rlk_adaln_gate_residual_fwd", "rlk_adaln_gate_residual_bwd",
    "rlk_adamw_step", "rlk_grad_norm", "rlk_grad_norm_workspace_bytes",
    "rlk_fp8_row_bytes", "rlk_fp8_scale_row_bytes", "rlk_fp8_quant_workspace_bytes", "rlk_fp8_quantize", "rlk_fp8_gemm",
    "rlk_muon_workspace_bytes", "rlk_muon_step", "rlk_orthogonalize",
)
OP_TRACE_CAP = 256
OP_TRACE_MAX_KERNELS = 8


class Shape(ctypes.Structure):
    """rlk_ja_shape."""
    _fields_ = [
        ("B", ctypes.c_int32), ("T_txt", ctypes.c_int32), ("grid_h", ctypes.c_int32),
        ("grid_w", ctypes.c_int32), ("H", ctypes.c_int32), ("D", ctypes.c_int32),
        ("eps", ctypes.c_float), ("theta", ctypes.c_float), ("axes", ctypes.c_int32 * 3),
    ]

    @classmethod
    def make(cls, B, T_txt, grid_h, grid_w, H, D=HEAD_DIM, eps=1e-6, theta=10000.0, axes=AXES):
        s = cls()
        s.B, s.T_txt, s.grid_h, s.grid_w, s.H, s.D = B, T_txt, grid_h, grid_w, H, D
        s.eps, s.theta = eps, theta
        s.axes[0], s.axes[1], s.axes[2] = axes
        return s

    @property
    def S(self) -> int:
        return self.T_txt + self.grid_h * self.grid_w


NORMS = {"none": 0, "layer": 1, "rms": 2}


class AdalnShape(ctypes.Structure):
    """rlk_adaln_shape."""
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T_txt", "T_img", "C", "norm", "post", "x_dtype", "y_dtype",
                                              "mod_dtype")] + \
               [("eps", ctypes.c_float), ("alpha", ctypes.c_float), ("mod_stride", ctypes.c_int64),
                ("dmod_stride", ctypes.c_int64)]

    @classmethod
    def make(cls, B, T_txt, T_img, C, norm="layer", post="none", x_fp32=False, y_fp32=False, mod_fp32=False, eps=1e-6,
             alpha=1.0, mod_stride=None, dmod_stride=None):
        return cls(B, T_txt, T_img, C, NORMS[norm], NORMS[post], int(x_fp32), int(y_fp32), int(mod_fp32), eps, alpha,
                   C if mod_stride is None else mod_stride, C if dmod_stride is None else dmod_stride)


class AdalnIo(ctypes.Structure):
    """rlk_adaln_io: one stream's buffers (device pointers)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "h", "gate", "scale", "shift", "w", "w_post", "r", "y", "stats",
                                               "post_stats")]


class AdalnGrad(ctypes.Structure):
    """rlk_adaln_grad: one stream's gradients (device pointers)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("dy", "dr", "dx", "dh", "dgate", "dscale", "dshift", "dw", "dw_post")]


class AdamwTensor(ctypes.Structure):
    """rlk_adamw_tensor."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "master", "g", "m", "v", "m_scale", "v_scale")] + \
               [("n", ctypes.c_int64), ("lr_scale", ctypes.c_double), ("weight_decay", ctypes.c_double),
                ("g_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32), ("key", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class AdamwArgs(ctypes.Structure):
    """rlk_adamw_args."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps")] + \
               [("step", ctypes.c_int64), ("lr_dev", ctypes.c_void_p), ("step_dev", ctypes.c_void_p),
                ("grad_scale", ctypes.c_void_p), ("seed", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


FP8_FORMATS = {"e4m3": 0, "e5m2": 1}
FP8_MAX_ITEMS, FP8_FEW_ROWS, FP8_FEW_K = 8, 16, 12288


class Fp8Quant(ctypes.Structure):
    """rlk_fp8_quant: one matrix to be rounded to codes."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "q", "q_scale", "qt", "qt_scale", "col_sum", "workspace")] + \
               [(n, ctypes.c_int64) for n in ("rows", "cols", "x_stride")] + \
               [(n, ctypes.c_int32) for n in ("x_dtype", "format", "square", "reserved")]


class Fp8Product(ctypes.Structure):
    """rlk_fp8_product: one product of two operands in codes."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("a", "a_scale", "b", "b_scale", "bias", "d")] + \
               [(n, ctypes.c_int64) for n in ("m", "n", "k", "d_stride")] + \
               [(n, ctypes.c_int32) for n in ("a_format", "b_format", "d_dtype", "accumulate", "a_rows", "reserved")]


class MuonMatrix(ctypes.Structure):
    """rlk_muon_matrix."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("p", "master", "g", "m")] + \
               [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("lr_scale", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("g_dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MuonArgs(ctypes.Structure):
    """rlk_muon_args."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "momentum", "update_rms", "a", "b", "c", "eps")] + \
               [("lr_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p), ("iterations", ctypes.c_int32),
                ("nesterov", ctypes.c_int32)]


class Trace(ctypes.Structure):
    """rlk_ja_trace."""
    _fields_ = [
        ("backend", ctypes.c_char * 32), ("reduction_order", ctypes.c_char * 160),
        ("accumulator", ctypes.c_char * 16), ("split_k", ctypes.c_int32),
        ("atomics", ctypes.c_int32), ("tf32", ctypes.c_int32), ("strict_math", ctypes.c_int32),
        ("block_q", ctypes.c_int32), ("block_kv", ctypes.c_int32),
        ("fingerprint", ctypes.c_char * 96),
    ]


class RlkError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({_strerror(code)})")


class OpRecord(ctypes.Structure):
    """rlk_op_record: one operator-trace record."""
    _fields_ = [
        ("seq", ctypes.c_uint64), ("op", ctypes.c_char * 48), ("entry_point", ctypes.c_char * 40),
        ("requested_backend", ctypes.c_char * 24), ("actual_backend", ctypes.c_char * 24),
        ("status", ctypes.c_int32), ("fallback", ctypes.c_int32), ("split_k", ctypes.c_int32),
        ("atomics", ctypes.c_int32), ("tf32", ctypes.c_int32), ("n_kernels", ctypes.c_int32),
        ("kernels", (ctypes.c_char * 32) * OP_TRACE_MAX_KERNELS), ("kernel_fingerprint", ctypes.c_char * 96),
        ("accumulator", ctypes.c_char * 16), ("arithmetic_policy", ctypes.c_char * 192),
        ("reduction_order", ctypes.c_char * 160), ("B", ctypes.c_int32), ("H", ctypes.c_int32),
        ("T_txt", ctypes.c_int32), ("grid_h", ctypes.c_int32), ("grid_w", ctypes.c_int32),
    ]

    def to_dict(self) -> dict:
        d = {}
        for f, _ in self._fields_:
            v = getattr(self, f)
            if f == "kernels":
                d[f] = [v[i].value.decode() for i in range(self.n_kernels)]
            elif isinstance(v, bytes):
                d[f] = v.decode()
            else:
                d[f] = v
        return d


_lib = None


def library_path() -> str:
    return os.path.join(_PKG, LIB_NAME)


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load a build of the library and declare its signatures."""
    path = path or library_path()
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`. "
            "There is no fallback implementation.")
    L = ctypes.CDLL(path)
    vp, sz, i32, f32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.POINTER(ctypes.c_float)
    shp = ctypes.POINTER(Shape)
    L.rlk_joint_attn_ctx_bytes.argtypes = [shp]
    L.rlk_joint_attn_ctx_bytes.restype = sz
    L.rlk_joint_attn_bwd_workspace_bytes.argtypes = [shp]
    L.rlk_joint_attn_bwd_workspace_bytes.restype = sz
    L.rlk_joint_attn_bwd_workspace_min_bytes.argtypes = [shp]
    L.rlk_joint_attn_bwd_workspace_min_bytes.restype = sz
    L.rlk_joint_attn_fwd.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(ctypes.c_int32),
                                     vp, vp, vp, vp]
    L.rlk_joint_attn_fwd.restype = i32
    L.rlk_joint_attn_bwd.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(ctypes.c_int32),
                                     vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.rlk_joint_attn_bwd.restype = i32
    L.rlk_joint_attn_check_status.argtypes = [vp]
    L.rlk_joint_attn_check_status.restype = i32
    L.rlk_strict_math_compiled.argtypes = []
    L.rlk_strict_math_compiled.restype = i32
    L.rlk_selftest_wait_timeout.argtypes = [i32, vp]
    L.rlk_selftest_wait_timeout.restype = i32
    L.rlk_fwd_tile_schedule.argtypes = [i32]
    L.rlk_fwd_tile_schedule.restype = i32
    L.rlk_joint_attn_trace.argtypes = [ctypes.POINTER(Trace)]
    L.rlk_joint_attn_trace.restype = i32
    L.rlk_strerror.argtypes = [i32]
    L.rlk_strerror.restype = ctypes.c_char_p
    L.rlk_kernel_timing.argtypes = [i32]
    L.rlk_kernel_timing.restype = i32
    L.rlk_kernel_timing_read.argtypes = [i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int32)]
    L.rlk_kernel_timing_read.restype = i32
    L.rlk_joint_attn_fwd_noalloc.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, ctypes.POINTER(ctypes.c_int32),
                                             vp, vp, vp]
    L.rlk_joint_attn_fwd_noalloc.restype = i32
    L.rlk_joint_attn_unfused_bytes.argtypes = [shp, i32]
    L.rlk_joint_attn_unfused_bytes.restype = sz
    L.rlk_qk_norm_rope.argtypes = [shp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.rlk_qk_norm_rope.restype = i32
    i32p = ctypes.POINTER(ctypes.c_int32)
    L.rlk_joint_attn_qk_gemm.argtypes = [shp, vp, i32p, vp, vp]
    L.rlk_joint_attn_qk_gemm.restype = i32
    L.rlk_joint_attn_softmax.argtypes = [shp, vp, i32p, vp, vp, vp, vp, vp]
    L.rlk_joint_attn_softmax.restype = i32
    L.rlk_joint_attn_av_gemm.argtypes = [shp, vp, vp, vp, vp, i32p, vp, vp]
    L.rlk_joint_attn_av_gemm.restype = i32
    L.rlk_joint_attn_bwd_stats.argtypes = [shp, vp, vp, vp, vp, vp]
    L.rlk_joint_attn_bwd_stats.restype = i32
    L.rlk_joint_attn_softmax_bwd.argtypes = [shp, vp, vp, vp, i32p, vp, vp, vp]
    L.rlk_joint_attn_softmax_bwd.restype = i32
    L.rlk_joint_attn_av_gemm_bwd.argtypes = [shp, vp, vp, vp, i32p, vp, vp, vp]
    L.rlk_joint_attn_av_gemm_bwd.restype = i32
    L.rlk_joint_attn_qk_gemm_bwd.argtypes = [shp, vp, vp, i32p, vp, vp, vp]
    L.rlk_joint_attn_qk_gemm_bwd.restype = i32
    L.rlk_qk_norm_rope_bwd.argtypes = [shp] + [vp] * 15
    L.rlk_qk_norm_rope_bwd.restype = i32
    L.rlk_joint_attn_state_bytes.argtypes = [shp]
    L.rlk_joint_attn_state_bytes.restype = sz
    L.rlk_joint_attn_fwd_shard.argtypes = [shp, vp, vp, i32p, ctypes.c_int32, ctypes.c_int32, vp, vp, vp, vp, vp]
    L.rlk_joint_attn_fwd_shard.restype = i32
    L.rlk_joint_attn_fwd_streams.argtypes = [shp] + [vp] * 10 + [i32p] + [vp] * 5
    L.rlk_joint_attn_fwd_streams.restype = i32
    L.rlk_joint_attn_bwd_streams.argtypes = [shp] + [vp] * 10 + [i32p] + [vp] * 14 + [sz, vp]
    L.rlk_joint_attn_bwd_streams.restype = i32
    L.rlk_qkv_bias_gemm.argtypes = [shp] + [vp] * 18
    L.rlk_qkv_bias_gemm.restype = i32
    L.rlk_joint_attn_fwd_ctx.argtypes = [shp, vp, vp, vp, i32p, vp, vp, vp, vp]
    L.rlk_joint_attn_fwd_ctx.restype = i32
    L.rlk_attn_out_bias_gemm.argtypes = [shp] + [vp] * 9
    L.rlk_attn_out_bias_gemm.restype = i32
    ash, aio, agr = ctypes.POINTER(AdalnShape), ctypes.POINTER(AdalnIo), ctypes.POINTER(AdalnGrad)
    L.rlk_adaln_workspace_bytes.argtypes = [ash]
    L.rlk_adaln_workspace_bytes.restype = sz
    for name in ("modulation", "gate_residual"):
        fwd, bwd = getattr(L, f"rlk_adaln_{name}_fwd"), getattr(L, f"rlk_adaln_{name}_bwd")
        fwd.argtypes, fwd.restype = [ash, aio, aio, vp], i32
        bwd.argtypes, bwd.restype = [ash, aio, aio, agr, agr, vp, sz, vp], i32
    adt = ctypes.POINTER(AdamwTensor)
    L.rlk_adamw_step.argtypes = [adt, ctypes.c_int32, ctypes.POINTER(AdamwArgs), vp]
    L.rlk_adamw_step.restype = i32
    L.rlk_grad_norm_workspace_bytes.argtypes = [adt, ctypes.c_int32]
    L.rlk_grad_norm_workspace_bytes.restype = sz
    L.rlk_grad_norm.argtypes = [adt, ctypes.c_int32, ctypes.c_float, ctypes.c_float, vp, vp, sz, vp]
    L.rlk_grad_norm.restype = i32
    i64 = ctypes.c_int64
    for name, args in (("row_bytes", [i64]), ("scale_row_bytes", [i64]), ("quant_workspace_bytes", [i64, i64])):
        f = getattr(L, "rlk_fp8_" + name)
        f.argtypes, f.restype = args, sz
    L.rlk_fp8_quantize.argtypes, L.rlk_fp8_quantize.restype = [ctypes.POINTER(Fp8Quant), ctypes.c_int32, vp], i32
    L.rlk_fp8_gemm.argtypes, L.rlk_fp8_gemm.restype = [ctypes.POINTER(Fp8Product), ctypes.c_int32, vp], i32
    mat = ctypes.POINTER(MuonMatrix)
    L.rlk_muon_workspace_bytes.argtypes, L.rlk_muon_workspace_bytes.restype = [mat, ctypes.c_int32], sz
    for name in ("rlk_muon_step", "rlk_orthogonalize"):
        f = getattr(L, name)
        f.argtypes, f.restype = [mat, ctypes.c_int32, ctypes.POINTER(MuonArgs), vp, sz, vp], i32
    L.rlk_op_trace_enable.argtypes = [i32]
    L.rlk_op_trace_enable.restype = i32
    L.rlk_op_trace_count.argtypes = []
    L.rlk_op_trace_count.restype = ctypes.c_int32
    L.rlk_op_trace_read.argtypes = [ctypes.c_int32, ctypes.POINTER(OpRecord)]
    L.rlk_op_trace_read.restype = i32
    return L


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = load_library()
    return _lib


def _strerror(code: int) -> str:
    try:
        return lib().rlk_strerror(code).decode()
    except Exception:  # the library itself failed to load
        return "?"


def _check(code: int, where: str) -> None:
    if code != RLK_OK:
        raise RlkError(code, where)


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream_handle(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _lengths(valid_len: Sequence[int], shape: Shape):
    """The host array of valid text lengths the C ABI reads: exactly B of
    them (the library reads B entries, so a shorter list is refused here)."""
    vals = [int(x) for x in valid_len]
    if len(vals) != shape.B:
        raise ValueError(f"expected {shape.B} valid text lengths (one per sample), got {len(vals)}")
    return (ctypes.c_int32 * max(1, len(vals)))(*vals)


def rlk_joint_attn_ctx_bytes(shape: Shape) -> int:
    return int(lib().rlk_joint_attn_ctx_bytes(ctypes.byref(shape)))


def rlk_joint_attn_bwd_workspace_bytes(shape: Shape) -> int:
    return int(lib().rlk_joint_attn_bwd_workspace_bytes(ctypes.byref(shape)))


def rlk_joint_attn_bwd_workspace_min_bytes(shape: Shape) -> int:
    return int(lib().rlk_joint_attn_bwd_workspace_min_bytes(ctypes.byref(shape)))


def rlk_joint_attn_fwd(shape, q, k, v, g_q_txt, g_k_txt, g_q_img, g_k_img, txt_valid_len,
                       out, lse, ctx, stream=None) -> None:
    """Enqueue the forward; tensors or raw device pointers (ints)."""
    rc = lib().rlk_joint_attn_fwd(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g_q_txt), _ptr(g_k_txt),
        _ptr(g_q_img), _ptr(g_k_img), _lengths(txt_valid_len, shape), _ptr(out), _ptr(lse), _ptr(ctx),
        _stream_handle(stream))
    _check(rc, "rlk_joint_attn_fwd")


def rlk_joint_attn_fwd_noalloc(shape, q, k, v, g_q_txt, g_k_txt, g_q_img, g_k_img, txt_valid_len,
                               out, lse, stream=None) -> None:
    """Enqueue the forward with the library's built-in device scratch (for
    callers that cannot allocate); forward-only, calls must not overlap."""
    rc = lib().rlk_joint_attn_fwd_noalloc(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g_q_txt), _ptr(g_k_txt),
        _ptr(g_q_img), _ptr(g_k_img), _lengths(txt_valid_len, shape), _ptr(out), _ptr(lse),
        _stream_handle(stream))
    _check(rc, "rlk_joint_attn_fwd_noalloc")


def rlk_joint_attn_bwd(shape, q, k, v, g_q_txt, g_k_txt, g_q_img, g_k_img, txt_valid_len,
                       out, dout, lse, ctx, dq, dk, dv, dg_partial, dg, workspace,
                       workspace_bytes=None, stream=None) -> None:
    """Enqueue the backward; tensors or raw device pointers (ints)."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib().rlk_joint_attn_bwd(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(g_q_txt), _ptr(g_k_txt),
        _ptr(g_q_img), _ptr(g_k_img), _lengths(txt_valid_len, shape), _ptr(out), _ptr(dout), _ptr(lse),
        _ptr(ctx), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg_partial), _ptr(dg), _ptr(workspace),
        int(workspace_bytes), _stream_handle(stream))
    _check(rc, "rlk_joint_attn_bwd")


def rlk_joint_attn_unfused_bytes(shape: Shape, which: str | int) -> int:
    w = UNFUSED[which] if isinstance(which, str) else int(which)
    return int(lib().rlk_joint_attn_unfused_bytes(ctypes.byref(shape), w))


def rlk_qk_norm_rope(shape, q, k, g_q_txt, g_k_txt, g_q_img, g_k_img, ctx, stream=None) -> None:
    """Enqueue qk_rmsnorm + multi_axis_rope into ctx."""
    rc = lib().rlk_qk_norm_rope(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(g_q_txt), _ptr(g_k_txt),
                                _ptr(g_q_img), _ptr(g_k_img), _ptr(ctx), _stream_handle(stream))
    _check(rc, "rlk_qk_norm_rope")


def rlk_joint_attn_qk_gemm(shape, ctx, txt_valid_len, scores, stream=None) -> None:
    rc = lib().rlk_joint_attn_qk_gemm(ctypes.byref(shape), _ptr(ctx), _lengths(txt_valid_len, shape), _ptr(scores),
                                      _stream_handle(stream))
    _check(rc, "rlk_joint_attn_qk_gemm")


def rlk_joint_attn_softmax(shape, scores, txt_valid_len, p, alpha, l, lse, stream=None) -> None:
    rc = lib().rlk_joint_attn_softmax(ctypes.byref(shape), _ptr(scores), _lengths(txt_valid_len, shape), _ptr(p),
                                      _ptr(alpha), _ptr(l), _ptr(lse), _stream_handle(stream))
    _check(rc, "rlk_joint_attn_softmax")


def rlk_joint_attn_av_gemm(shape, p, alpha, l, v, txt_valid_len, out, stream=None) -> None:
    rc = lib().rlk_joint_attn_av_gemm(ctypes.byref(shape), _ptr(p), _ptr(alpha), _ptr(l), _ptr(v),
                                      _lengths(txt_valid_len, shape), _ptr(out), _stream_handle(stream))
    _check(rc, "rlk_joint_attn_av_gemm")


def rlk_joint_attn_bwd_stats(shape, out, dout, lse, stats, stream=None) -> None:
    _check(lib().rlk_joint_attn_bwd_stats(ctypes.byref(shape), _ptr(out), _ptr(dout), _ptr(lse), _ptr(stats),
                                          _stream_handle(stream)), "rlk_joint_attn_bwd_stats")


def rlk_joint_attn_softmax_bwd(shape, scores, stats, dp, txt_valid_len, p, ds, stream=None) -> None:
    _check(lib().rlk_joint_attn_softmax_bwd(ctypes.byref(shape), _ptr(scores), _ptr(stats), _ptr(dp),
                                            _lengths(txt_valid_len, shape), _ptr(p), _ptr(ds),
                                            _stream_handle(stream)), "rlk_joint_attn_softmax_bwd")


def rlk_joint_attn_av_gemm_bwd(shape, p, v, dout, txt_valid_len, dv, dp, stream=None) -> None:
    _check(lib().rlk_joint_attn_av_gemm_bwd(ctypes.byref(shape), _ptr(p), _ptr(v), _ptr(dout),
                                            _lengths(txt_valid_len, shape), _ptr(dv), _ptr(dp),
                                            _stream_handle(stream)), "rlk_joint_attn_av_gemm_bwd")


def rlk_joint_attn_qk_gemm_bwd(shape, ds, ctx, txt_valid_len, dqh, dkh, stream=None) -> None:
    _check(lib().rlk_joint_attn_qk_gemm_bwd(ctypes.byref(shape), _ptr(ds), _ptr(ctx),
                                            _lengths(txt_valid_len, shape), _ptr(dqh), _ptr(dkh),
                                            _stream_handle(stream)), "rlk_joint_attn_qk_gemm_bwd")


def rlk_qk_norm_rope_bwd(shape, q, k, g_q_txt, g_k_txt, g_q_img, g_k_img, ctx, dqh, dkh, dq, dk, dg_partial, dg,
                         gain_tiles, stream=None) -> None:
    _check(lib().rlk_qk_norm_rope_bwd(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(g_q_txt), _ptr(g_k_txt),
                                      _ptr(g_q_img), _ptr(g_k_img), _ptr(ctx), _ptr(dqh), _ptr(dkh), _ptr(dq),
                                      _ptr(dk), _ptr(dg_partial), _ptr(dg), _ptr(gain_tiles),
                                      _stream_handle(stream)), "rlk_qk_norm_rope_bwd")


def rlk_joint_attn_state_bytes(shape: Shape) -> int:
    return int(lib().rlk_joint_attn_state_bytes(ctypes.byref(shape)))


def rlk_joint_attn_fwd_shard(shape, ctx, v, txt_valid_len, blk_begin, blk_end, state_in, state_out, out, lse,
                             stream=None) -> None:
    """Enqueue the forward over key column blocks [blk_begin, blk_end),
    handing the online-softmax state on (see the header)."""
    rc = lib().rlk_joint_attn_fwd_shard(ctypes.byref(shape), _ptr(ctx), _ptr(v), _lengths(txt_valid_len, shape),
                                        int(blk_begin), int(blk_end), _ptr(state_in), _ptr(state_out), _ptr(out),
                                        _ptr(lse), _stream_handle(stream))
    _check(rc, "rlk_joint_attn_fwd_shard")


def rlk_joint_attn_fwd_streams(shape, q, k, v, g_q_txt, g_k_txt, g_q_img, g_k_img, txt_valid_len, out, lse, ctx,
                               stream=None) -> None:
    """Forward on separate streams: q, k, v and out are (text, image) pairs
    of tensors or device pointers (the text one may be None if T_txt == 0)."""
    args = [_ptr(x) for pair in (q, k, v) for x in pair]
    rc = lib().rlk_joint_attn_fwd_streams(
        ctypes.byref(shape), *args, _ptr(g_q_txt), _ptr(g_k_txt), _ptr(g_q_img), _ptr(g_k_img),
        _lengths(txt_valid_len, shape), _ptr(out[0]), _ptr(out[1]), _ptr(lse), _ptr(ctx), _stream_handle(stream))
    _check(rc, "rlk_joint_attn_fwd_streams")


def rlk_joint_attn_bwd_streams(shape, q, k, v, g_q_txt, g_k_txt, g_q_img, g_k_img, txt_valid_len, out, dout, lse,
                               ctx, dq, dk, dv, dg_partial, dg, workspace, workspace_bytes=None, stream=None) -> None:
    """Backward on separate streams; activations as (text, image) pairs."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    ins = [_ptr(x) for pair in (q, k, v) for x in pair]
    rc = lib().rlk_joint_attn_bwd_streams(
        ctypes.byref(shape), *ins, _ptr(g_q_txt), _ptr(g_k_txt), _ptr(g_q_img), _ptr(g_k_img),
        _lengths(txt_valid_len, shape), _ptr(out[0]), _ptr(out[1]), _ptr(dout[0]), _ptr(dout[1]), _ptr(lse), _ptr(ctx),
        _ptr(dq[0]), _ptr(dq[1]), _ptr(dk[0]), _ptr(dk[1]), _ptr(dv[0]), _ptr(dv[1]), _ptr(dg_partial), _ptr(dg),
        _ptr(workspace), int(workspace_bytes), _stream_handle(stream))
    _check(rc, "rlk_joint_attn_bwd_streams")


def rlk_qkv_bias_gemm(shape, x, w, b, gains, ctx, q, k, v, stream=None) -> None:
    """Per-stream QKV projection; x, w, b, q, k, v are (text, image) pairs
    (q, k may be (None, None) when ctx is given); gains a [4, 128] tensor or
    None (plain mode, ctx None)."""
    g = [None] * 4 if gains is None else [gains[0], gains[1], gains[2], gains[3]]
    rc = lib().rlk_qkv_bias_gemm(
        ctypes.byref(shape), _ptr(x[0]), _ptr(x[1]), _ptr(w[0]), _ptr(w[1]), _ptr(b[0]), _ptr(b[1]),
        *[_ptr(t) for t in g], _ptr(ctx), _ptr(q[0]), _ptr(q[1]), _ptr(k[0]), _ptr(k[1]), _ptr(v[0]), _ptr(v[1]),
        _stream_handle(stream))
    _check(rc, "rlk_qkv_bias_gemm")


def rlk_joint_attn_fwd_ctx(shape, ctx, v, txt_valid_len, out, lse, stream=None) -> None:
    """Attention from a prepared context; v and out are (text, image) pairs."""
    rc = lib().rlk_joint_attn_fwd_ctx(ctypes.byref(shape), _ptr(ctx), _ptr(v[0]), _ptr(v[1]),
                                      _lengths(txt_valid_len, shape), _ptr(out[0]), _ptr(out[1]), _ptr(lse),
                                      _stream_handle(stream))
    _check(rc, "rlk_joint_attn_fwd_ctx")


def rlk_attn_out_bias_gemm(shape, o, w, b, y, stream=None) -> None:
    """Per-stream output projection; o, w, b, y are (text, image) pairs."""
    rc = lib().rlk_attn_out_bias_gemm(ctypes.byref(shape), _ptr(o[0]), _ptr(o[1]), _ptr(w[0]), _ptr(w[1]),
                                      _ptr(b[0]), _ptr(b[1]), _ptr(y[0]), _ptr(y[1]), _stream_handle(stream))
    _check(rc, "rlk_attn_out_bias_gemm")


def rlk_adaln_workspace_bytes(shape: AdalnShape) -> int:
    return int(lib().rlk_adaln_workspace_bytes(ctypes.byref(shape)))


def _ref(struct):
    return None if struct is None else ctypes.byref(struct)


def rlk_adaln_modulation_fwd(shape, io, stream=None) -> None:
    """Enqueue adaln_modulation; io is a (text, image) pair of AdalnIo (None
    for a stream without tokens)."""
    _check(lib().rlk_adaln_modulation_fwd(_ref(shape), _ref(io[0]), _ref(io[1]), _stream_handle(stream)),
           "rlk_adaln_modulation_fwd")


def rlk_adaln_gate_residual_fwd(shape, io, stream=None) -> None:
    """Enqueue adaln_gate_residual with the next adaln_modulation."""
    _check(lib().rlk_adaln_gate_residual_fwd(_ref(shape), _ref(io[0]), _ref(io[1]), _stream_handle(stream)),
           "rlk_adaln_gate_residual_fwd")


def rlk_adaln_modulation_bwd(shape, io, grad, workspace, workspace_bytes=None, stream=None) -> None:
    """Enqueue the modulation's backward; io and grad are (text, image) pairs."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().rlk_adaln_modulation_bwd(_ref(shape), _ref(io[0]), _ref(io[1]), _ref(grad[0]), _ref(grad[1]),
                                          _ptr(workspace), int(workspace_bytes), _stream_handle(stream)),
           "rlk_adaln_modulation_bwd")


def rlk_adaln_gate_residual_bwd(shape, io, grad, workspace, workspace_bytes=None, stream=None) -> None:
    """Enqueue the gate-residual's backward; io and grad are (text, image) pairs."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().rlk_adaln_gate_residual_bwd(_ref(shape), _ref(io[0]), _ref(io[1]), _ref(grad[0]), _ref(grad[1]),
                                             _ptr(workspace), int(workspace_bytes), _stream_handle(stream)),
           "rlk_adaln_gate_residual_bwd")


def rlk_adamw_step(tensors, n_tensors, args, stream=None) -> None:
    """Enqueue one AdamW step over an array of AdamwTensor."""
    _check(lib().rlk_adamw_step(tensors, int(n_tensors), _ref(args), _stream_handle(stream)), "rlk_adamw_step")


def rlk_grad_norm_workspace_bytes(tensors, n_tensors) -> int:
    return int(lib().rlk_grad_norm_workspace_bytes(tensors, int(n_tensors)))


def rlk_grad_norm(tensors, n_tensors, pre_scale, max_norm, out, workspace, workspace_bytes=None, stream=None) -> None:
    """Enqueue the list's gradient norm and clip factor into out [2]."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib().rlk_grad_norm(tensors, int(n_tensors), float(pre_scale), float(max_norm), _ptr(out), _ptr(workspace),
                               int(workspace_bytes), _stream_handle(stream)), "rlk_grad_norm")


def rlk_op_trace_enable(enable: bool) -> None:
    _check(lib().rlk_op_trace_enable(1 if enable else 0), "rlk_op_trace_enable")


def rlk_op_trace_count() -> int:
    return int(lib().rlk_op_trace_count())


def rlk_op_trace_read() -> list[dict]:
    """Every record kept, oldest first, as dicts."""
    out = []
    for i in range(rlk_op_trace_count()):
        r = OpRecord()
        _check(lib().rlk_op_trace_read(i, ctypes.byref(r)), "rlk_op_trace_read")
        out.append(r.to_dict())
    return out


class op_trace:
    """Context manager: records every library call made inside it.
    ``with op_trace() as t: ...``; afterwards ``t.records`` holds the records."""

    def __enter__(self):
        rlk_op_trace_enable(True)
        self.records = []
        return self

    def __exit__(self, *exc):
        self.records = rlk_op_trace_read()
        rlk_op_trace_enable(False)
        return False


def rlk_joint_attn_check_status(stream=None) -> None:
    _check(lib().rlk_joint_attn_check_status(_stream_handle(stream)), "rlk_joint_attn_check_status")


def rlk_strict_math_compiled() -> int:
    return int(lib().rlk_strict_math_compiled())


def rlk_selftest_wait_timeout(limit_ms: int, stream=None) -> None:
    """Enqueue one warp whose bounded wait on a barrier nothing completes
    gives up after limit_ms: the next rlk_joint_attn_check_status() raises
    RlkError(RLK_ERR_DEVICE_TIMEOUT)."""
    _check(lib().rlk_selftest_wait_timeout(int(limit_ms), _stream_handle(stream)), "rlk_selftest_wait_timeout")


def rlk_joint_attn_trace() -> dict:
    t = Trace()
    _check(lib().rlk_joint_attn_trace(ctypes.byref(t)), "rlk_joint_attn_trace")
    return {f: (getattr(t, f).decode() if isinstance(getattr(t, f), bytes) else getattr(t, f))
            for f, _ in Trace._fields_}


FWD_TILES = {"auto": 0, "pairs": 1, "single": 2}


def rlk_fwd_tile_schedule(policy: str) -> str:
    """Set the fused forward's query-tile schedule ("auto", "pairs" or
    "single"; time only, never bytes); returns the previous one."""
    if policy not in FWD_TILES:
        raise ValueError(f"unknown tile schedule {policy!r}")
    prev = lib().rlk_fwd_tile_schedule(FWD_TILES[policy])
    if prev < 0:
        raise RuntimeError("rlk_fwd_tile_schedule refused the policy")
    return {v: k for k, v in FWD_TILES.items()}[prev]


def rlk_fp8_row_bytes(k: int) -> int:
    return lib().rlk_fp8_row_bytes(k)


def rlk_fp8_scale_row_bytes(k: int) -> int:
    return lib().rlk_fp8_scale_row_bytes(k)


def rlk_fp8_quant_workspace_bytes(rows: int, cols: int) -> int:
    return lib().rlk_fp8_quant_workspace_bytes(rows, cols)


def rlk_fp8_quantize(items, stream=None) -> None:
    """items: a ctypes array of Fp8Quant."""
    _check(lib().rlk_fp8_quantize(items, len(items), _stream_handle(stream)), "rlk_fp8_quantize")


def rlk_fp8_gemm(items, stream=None) -> None:
    """items: a ctypes array of Fp8Product."""
    _check(lib().rlk_fp8_gemm(items, len(items), _stream_handle(stream)), "rlk_fp8_gemm")


def rlk_muon_workspace_bytes(matrices) -> int:
    """matrices: a ctypes array of MuonMatrix."""
    return lib().rlk_muon_workspace_bytes(matrices, len(matrices))


def rlk_muon_step(matrices, args: MuonArgs, workspace, stream=None) -> None:
    _check(lib().rlk_muon_step(matrices, len(matrices), ctypes.byref(args), _ptr(workspace), workspace.numel(),
                               _stream_handle(stream)), "rlk_muon_step")


def rlk_orthogonalize(matrices, args: MuonArgs, workspace, stream=None) -> None:
    _check(lib().rlk_orthogonalize(matrices, len(matrices), ctypes.byref(args), _ptr(workspace), workspace.numel(),
                                   _stream_handle(stream)), "rlk_orthogonalize")


def rlk_strerror(code: int) -> str:
    return _strerror(code)


def rlk_kernel_timing(enable: bool) -> None:
    _check(lib().rlk_kernel_timing(1 if enable else 0), "rlk_kernel_timing")


def rlk_kernel_timing_read(kernel: str | int) -> tuple[float, int]:
    kid = KERNEL_IDS[kernel] if isinstance(kernel, str) else int(kernel)
    ms, n = ctypes.c_double(), ctypes.c_int32()
    _check(lib().rlk_kernel_timing_read(kid, ctypes.byref(ms), ctypes.byref(n)), "rlk_kernel_timing_read")
    return ms.value, n.value


class JointAttention:
    """Buffers + calls for one geometry: allocates the caller-owned tensors
    with PyTorch and passes them to the C ABI. Inputs are bf16 [B, S, H, 128]
    CUDA tensors; gains a float32 [4, 128] tensor (q_txt, k_txt, q_img, k_img)."""

    def __init__(self, B: int, T_txt: int, grid_h: int, grid_w: int, H: int, device="cuda",
                 eps: float = 1e-6, theta: float = 10000.0, ws_budget_bytes: int | None = None):
        """ws_budget_bytes caps the backward workspace: with less than the
        full size the backward runs its (sample, head) pairs in groups (same
        bytes, more launches); below the minimum it raises."""
        import torch
        self.shape = Shape.make(B, T_txt, grid_h, grid_w, H, eps=eps, theta=theta)
        self.device = torch.device(device)
        n_ctx = rlk_joint_attn_ctx_bytes(self.shape)
        n_ws = rlk_joint_attn_bwd_workspace_bytes(self.shape)
        if n_ctx == 0 or n_ws == 0:
            raise RlkError(1, "JointAttention: invalid shape")
        if ws_budget_bytes is not None:
            n_min = rlk_joint_attn_bwd_workspace_min_bytes(self.shape)
            if ws_budget_bytes < n_min:
                raise RlkError(4, f"JointAttention: workspace budget {ws_budget_bytes} below the minimum {n_min}")
            n_ws = min(n_ws, int(ws_budget_bytes))
        self.ctx = torch.empty(n_ctx, dtype=torch.uint8, device=self.device)
        self.workspace = torch.empty(n_ws, dtype=torch.uint8, device=self.device)

    def _check_inputs(self, *ts):
        import torch
        sh = self.shape
        want = (sh.B, sh.S, sh.H, HEAD_DIM)
        for t in ts:
            if t.dtype != torch.bfloat16 or tuple(t.shape) != want or not t.is_contiguous() or t.device != self.device:
                raise ValueError(f"expected contiguous bf16 {want} on {self.device}, got {t.dtype} "
                                 f"{tuple(t.shape)} on {t.device}")

    def _check_f32(self, t, want, name):
        import torch
        if t.dtype != torch.float32 or tuple(t.shape) != tuple(want) or not t.is_contiguous() \
                or t.device != self.device:
            raise ValueError(f"{name} must be a contiguous float32 {tuple(want)} tensor on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")

    def _check_gains(self, gains):
        import torch
        if gains.dtype != torch.float32 or tuple(gains.shape) != (4, HEAD_DIM) or not gains.is_contiguous() \
                or gains.device != self.device:
            raise ValueError("gains must be a contiguous float32 [4, 128] tensor on the device")

    def forward(self, q, k, v, gains, valid_len, out=None, lse=None, want_lse=True, stream=None):
        import torch
        self._check_inputs(q, k, v)
        self._check_gains(gains)
        if len(valid_len) != self.shape.B:
            raise ValueError("one valid length per sample")
        sh = self.shape
        if out is None:
            out = torch.empty_like(q)
        else:
            self._check_inputs(out)
        if lse is None and want_lse:
            lse = torch.empty((sh.B, sh.H, sh.S), dtype=torch.float32, device=self.device)
        elif lse is not None:
            self._check_f32(lse, (sh.B, sh.H, sh.S), "lse")
        rlk_joint_attn_fwd(self.shape, q, k, v, gains[0], gains[1], gains[2], gains[3], valid_len,
                           out, lse, self.ctx, stream)
        return out, lse

    def backward(self, q, k, v, gains, valid_len, out, dout, lse, dq=None, dk=None, dv=None,
                 dg_partial=None, dg=None, stream=None):
        import torch
        self._check_inputs(q, k, v, out, dout)
        self._check_gains(gains)
        sh = self.shape
        self._check_f32(lse, (sh.B, sh.H, sh.S), "lse")
        dq = torch.empty_like(q) if dq is None else dq
        dk = torch.empty_like(k) if dk is None else dk
        dv = torch.empty_like(v) if dv is None else dv
        self._check_inputs(dq, dk, dv)
        if dg_partial is None:
            dg_partial = torch.empty((sh.B, sh.H, 4, HEAD_DIM), dtype=torch.float32, device=self.device)
        if dg is None:
            dg = torch.empty((4, HEAD_DIM), dtype=torch.float32, device=self.device)
        self._check_f32(dg_partial, (sh.B, sh.H, 4, HEAD_DIM), "dg_partial")
        self._check_f32(dg, (4, HEAD_DIM), "dg")
        rlk_joint_attn_bwd(sh, q, k, v, gains[0], gains[1], gains[2], gains[3], valid_len, out, dout,
                           lse, self.ctx, dq, dk, dv, dg_partial, dg, self.workspace, stream=stream)
        return dq, dk, dv, dg_partial, dg

    def forward_unfused(self, q, k, v, gains, valid_len, stream=None):
        """The forward as the four standalone operators (qk_rmsnorm +
        multi_axis_rope, joint_attn_qk_gemm, joint_attn_softmax,
        joint_attn_av_gemm) with materialised intermediates. Returns a dict
        with out, lse and the intermediates scores [B, H, S, n_tiles*128]
        fp32, p (same shape, bf16), alpha [B, H, S, n_tiles] fp32 and l."""
        import torch
        self._check_inputs(q, k, v)
        self._check_gains(gains)
        if len(valid_len) != self.shape.B:
            raise ValueError("one valid length per sample")
        sh = self.shape
        n_tiles = -(-sh.T_txt // 128) + -(-(sh.grid_h * sh.grid_w) // 128)
        dev = self.device
        scores = torch.empty((sh.B, sh.H, sh.S, n_tiles * 128), dtype=torch.float32, device=dev)
        p = torch.empty((sh.B, sh.H, sh.S, n_tiles * 128), dtype=torch.bfloat16, device=dev)
        alpha = torch.empty((sh.B, sh.H, sh.S, n_tiles), dtype=torch.float32, device=dev)
        l = torch.empty((sh.B, sh.H, sh.S), dtype=torch.float32, device=dev)
        lse = torch.empty((sh.B, sh.H, sh.S), dtype=torch.float32, device=dev)
        out = torch.empty_like(q)
        rlk_qk_norm_rope(sh, q, k, gains[0], gains[1], gains[2], gains[3], self.ctx, stream)
        rlk_joint_attn_qk_gemm(sh, self.ctx, valid_len, scores, stream)
        rlk_joint_attn_softmax(sh, scores, valid_len, p, alpha, l, lse, stream)
        rlk_joint_attn_av_gemm(sh, p, alpha, l, v, valid_len, out, stream)
        return {"out": out, "lse": lse, "l": l, "scores": scores, "p": p, "alpha": alpha}

    def backward_unfused(self, q, k, v, gains, valid_len, out, dout, lse, scores, stream=None):
        """The backward as the standalone operators' backward calls, after a
        forward (fused or standalone) on the same inputs left its context in
        this object; scores from rlk_joint_attn_qk_gemm. Returns a dict with
        dq, dk, dv, dgp, dg (bytes equal to backward()) and the intermediates
        stats, p, dp, ds, dqh, dkh."""
        import torch
        self._check_inputs(q, k, v, out, dout)
        self._check_gains(gains)
        if len(valid_len) != self.shape.B:
            raise ValueError("one valid length per sample")
        sh = self.shape
        n_tiles = -(-sh.T_txt // 128) + -(-(sh.grid_h * sh.grid_w) // 128)
        dev = self.device
        stats = torch.empty((2, sh.B, sh.H, n_tiles * 128), dtype=torch.float32, device=dev)
        p = torch.empty((sh.B, sh.H, sh.S, n_tiles * 128), dtype=torch.bfloat16, device=dev)
        ds = torch.empty_like(p)
        dp = torch.empty((sh.B, sh.H, sh.S, n_tiles * 128), dtype=torch.float32, device=dev)
        dqh = torch.empty((sh.B, sh.H, sh.S, HEAD_DIM), dtype=torch.float32, device=dev)
        dkh = torch.empty_like(dqh)
        gain_tiles = torch.empty(rlk_joint_attn_unfused_bytes(sh, UNFUSED["gain_tiles"]) // 4, dtype=torch.float32,
                                 device=dev)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        dgp = torch.empty((sh.B, sh.H, 4, HEAD_DIM), dtype=torch.float32, device=dev)
        dg = torch.empty((4, HEAD_DIM), dtype=torch.float32, device=dev)
        rlk_joint_attn_bwd_stats(sh, out, dout, lse, stats, stream)
        rlk_joint_attn_softmax_bwd(sh, scores, stats, None, valid_len, p, None, stream)
        rlk_joint_attn_av_gemm_bwd(sh, p, v, dout, valid_len, dv, dp, stream)
        rlk_joint_attn_softmax_bwd(sh, scores, stats, dp, valid_len, None, ds, stream)
        rlk_joint_attn_qk_gemm_bwd(sh, ds, self.ctx, valid_len, dqh, dkh, stream)
        rlk_qk_norm_rope_bwd(sh, q, k, gains[0], gains[1], gains[2], gains[3], self.ctx, dqh, dkh, dq, dk, dgp, dg,
                             gain_tiles, stream)
        return {"dq": dq, "dk": dk, "dv": dv, "dgp": dgp, "dg": dg, "stats": stats, "p": p, "dp": dp, "ds": ds,
                "dqh": dqh, "dkh": dkh}

    def forward_streams(self, q, k, v, gains, valid_len, stream=None):
        """Forward on separate text/image tensors: q, k, v are (txt, img)
        pairs, txt [B, T_txt, H, 128] and img [B, grid_h*grid_w, H, 128]
        bf16. Returns ((out_txt, out_img), lse)."""
        import torch
        sh = self.shape
        out = tuple(None if x is None else torch.empty_like(x) for x in q)
        lse = torch.empty((sh.B, sh.H, sh.S), dtype=torch.float32, device=self.device)
        rlk_joint_attn_fwd_streams(sh, q, k, v, gains[0], gains[1], gains[2], gains[3], valid_len, out, lse,
                                   self.ctx, stream)
        return out, lse

    def backward_streams(self, q, k, v, gains, valid_len, out, dout, lse, stream=None):
        """Backward on separate text/image tensors (pairs as in
        forward_streams). Returns dq, dk, dv pairs, dg_partial and dg."""
        import torch
        sh = self.shape
        like = lambda pair: tuple(None if x is None else torch.empty_like(x) for x in pair)  # noqa: E731
        dq, dk, dv = like(q), like(k), like(v)
        dgp = torch.empty((sh.B, sh.H, 4, HEAD_DIM), dtype=torch.float32, device=self.device)
        dg = torch.empty((4, HEAD_DIM), dtype=torch.float32, device=self.device)
        rlk_joint_attn_bwd_streams(sh, q, k, v, gains[0], gains[1], gains[2], gains[3], valid_len, out, dout, lse,
                                   self.ctx, dq, dk, dv, dgp, dg, self.workspace, stream=stream)
        return dq, dk, dv, dgp, dg

    def n_key_blocks(self) -> int:
        sh = self.shape
        return -(-sh.T_txt // 128) + -(-(sh.grid_h * sh.grid_w) // 128)

    def forward_sharded(self, q, k, v, gains, valid_len, bounds, stream=None):
        """The forward run as consecutive key shards handing the softmax
        state on (ring order). ``bounds`` are the shard boundaries inside
        (0, n_key_blocks()), ascending. Returns out and lse."""
        import torch
        self._check_inputs(q, k, v)
        self._check_gains(gains)
        sh = self.shape
        edges = [0] + [int(x) for x in bounds] + [self.n_key_blocks()]
        out = torch.empty_like(q)
        lse = torch.empty((sh.B, sh.H, sh.S), dtype=torch.float32, device=self.device)
        n_state = rlk_joint_attn_state_bytes(sh) // 4
        states = [torch.empty(n_state, dtype=torch.float32, device=self.device) for _ in range(2)]
        rlk_qk_norm_rope(sh, q, k, gains[0], gains[1], gains[2], gains[3], self.ctx, stream)
        for i in range(len(edges) - 1):
            last = i == len(edges) - 2
            st_in = None if i == 0 else states[(i - 1) % 2]
            st_out = None if last else states[i % 2]
            rlk_joint_attn_fwd_shard(sh, self.ctx, v, valid_len, edges[i], edges[i + 1], st_in, st_out,
                                     out if last else None, lse if last else None, stream)
        return out, lse

    def ctx_views(self):
        """Views of the forward context: qh, kh bf16 [B, H, S, 128]; rq, rk fp32 [B, H, S].
        The offsets follow the library's ctx layout (regions aligned to 256 bytes)."""
        import torch
        sh = self.shape
        rows = sh.B * sh.H * sh.S

        def up(x):
            return (x + 255) // 256 * 256
        o_kh = up(rows * HEAD_DIM * 2)
        o_rq = up(o_kh + rows * HEAD_DIM * 2)
        o_rk = up(o_rq + rows * 4)
        c = self.ctx
        qh = c[:rows * HEAD_DIM * 2].view(torch.bfloat16).view(sh.B, sh.H, sh.S, HEAD_DIM)
        kh = c[o_kh:o_kh + rows * HEAD_DIM * 2].view(torch.bfloat16).view(sh.B, sh.H, sh.S, HEAD_DIM)
        rq = c[o_rq:o_rq + rows * 4].view(torch.float32).view(sh.B, sh.H, sh.S)
        rk = c[o_rk:o_rk + rows * 4].view(torch.float32).view(sh.B, sh.H, sh.S)
        return qh, kh, rq, rk


def _require_current(device) -> None:
    """The library launches on the current device: it must be the tensors' one."""
    import torch
    if device.type != "cuda":
        raise ValueError(f"the buffers are on {device}: the library computes on CUDA devices only")
    if torch._C._cuda_getDevice() != device.index:
        raise ValueError(f"the current device is cuda:{torch.cuda.current_device()}, the buffers are on {device}")


def _raw_stream(stream, index) -> int:
    """The handle of `stream`, or of device `index`'s current one without
    making a torch.cuda.Stream of it (3 us a call)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(index)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _empty(size, dtype, device, stream):
    """Memory for a call on `stream`: what the allocator hands out for a stream
    is free there, and maybe not yet on another one."""
    import torch
    if stream is None:
        return torch.empty(size, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream):
        return torch.empty(size, dtype=dtype, device=device)


def _workspace(owner, size, stream, handle):
    """The workspace of an object's calls, allocated at the first one. Its memory
    goes back to the stream it was allocated for when the object does, perhaps
    while another stream's call still works in it: a torch stream that uses it is
    recorded, so that the memory waits for it."""
    import torch
    if owner.workspace is None:
        owner.workspace = _empty(size, torch.uint8, owner.device, stream)
        owner._streams = {handle}
    elif handle not in owner._streams and owner.workspace.is_cuda:
        s = torch.cuda.current_stream(owner.device) if stream is None else stream
        if not isinstance(s, int):
            owner.workspace.record_stream(s)
        owner._streams.add(handle)
    return owner.workspace


_NONE = (None, None)


class _Results(dict):
    """What a call returned, with its pointers: passed back as ``out`` of the
    same kind of call, it is looked at only for holding the same memory still
    (checking seven pairs anew takes longer than the smallest kernels)."""

    def __init__(self, kinds, names, pairs, pointers):
        super().__init__(pairs)
        self.kinds, self.names, self.pairs, self.pointers = kinds, names, list(pairs.values()), pointers
        self.tensors = [t for pair in self.pairs for t in pair if t is not None]
        self.addresses = [t.data_ptr() for t in self.tensors]
        # (held, so that no other memory can come to these addresses)
        self.storages = [t.untyped_storage() for t in self.tensors]

    def fits(self, kinds, names):
        return self.kinds is kinds and self.names == names and len(self) == len(self.pairs) and \
            all(map(operator.is_, self.values(), self.pairs)) and [t.data_ptr() for t in self.tensors] == self.addresses


class _Pairs:
    """Checks and outputs of calls on (text, image) pairs of tensors: a subclass has ``device``, ``_index`` and, for
    each output, ``_kinds``: its sizes (None where a stream has no tokens) and type."""

    def _bad(self, name, i, t, want, dtype):
        if want is None:
            raise ValueError(f"{name}[{i}] must be None: the stream has no tokens")
        if t is None:
            raise ValueError(f"{name}[{i}] is missing")
        raise ValueError(f"{name}[{i}] must be a contiguous {dtype} {tuple(want)} tensor on {self.device}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")

    def _need(self, name, pair, dtype, sizes):
        """Pointers of a pair of required dense tensors (None without tokens)."""
        if len(pair) != 2:
            raise ValueError(f"{name} must be a (text, image) pair")
        index = self._index
        t, want = pair[0], sizes[0]
        p = q = None
        if t is not None:
            if want is None or t.dtype is not dtype or t.shape != want or not t.is_contiguous() or t.get_device() != index:
                self._bad(name, 0, t, want, dtype)
            p = t.data_ptr()
        elif want is not None:
            self._bad(name, 0, t, want, dtype)
        t, want = pair[1], sizes[1]
        if t is not None:
            if want is None or t.dtype is not dtype or t.shape != want or not t.is_contiguous() or t.get_device() != index:
                self._bad(name, 1, t, want, dtype)
            q = t.data_ptr()
        elif want is not None:
            self._bad(name, 1, t, want, dtype)
        return p, q

    def _outputs(self, out, names, stream):
        """The outputs of these names, new or taken from `out`, and their pointers."""
        of = self._kinds
        if type(out) is _Results and out.fits(of, names):
            return out, out.pointers
        if out is None:
            pairs = {k: tuple(None if s is None else _empty(s, of[k][1], self.device, stream) for s in of[k][0])
                     for k in names}
            out = _Results(of, names, pairs, {k: self._need(k, pairs[k], of[k][1], of[k][0]) for k in names})
            return out, out.pointers
        if len(out) != len(names) or any(k not in out for k in names):
            raise ValueError(f"out must hold {sorted(names)}, got {sorted(out)}")
        return out, {k: self._need(k, out[k], of[k][1], of[k][0]) for k in names}


class AdaLN(_Pairs):
    """Buffers + calls of the block's norms, modulation, gate and residual for
    one geometry: adaln_modulation before a sublayer's projections,
    adaln_gate_residual (with the next modulation) after them.

    Activations are (text, image) pairs, [B, T_txt, C] and [B, T_img, C], a
    pair's text None if T_txt is 0 and its image None if T_img is 0.
    ``scale``, ``shift`` and ``gate`` are pairs of [B, C] views (columns of the
    modulation projection's output, all with one sample stride) or None (0, 0
    and 1). ``w`` and ``w_post`` are pairs of float32 [C] norm weights or None.
    x, r and their gradients have ``x_dtype``; y, h and theirs ``y_dtype``.

    Every call returns its outputs as a dict of pairs; passing that dict back
    as ``out`` reuses its buffers. The backward calls share one workspace:
    calls that may overlap on the GPU (other streams, graphs replayed at the
    same time) need an object each. An object outlives the graphs that captured
    its calls, and its calls on a stream that is given as an address."""

    def __init__(self, B: int, T_txt: int, T_img: int, C: int, norm: str = "layer", post: str | None = None,
                 x_dtype=None, y_dtype=None, mod_dtype=None, eps: float = 1e-6, alpha: float = 1.0, device="cuda"):
        import torch
        bf16, f32 = torch.bfloat16, torch.float32
        self.x_dtype, self.y_dtype, self.mod_dtype = x_dtype or bf16, y_dtype or bf16, mod_dtype or bf16
        if not {self.x_dtype, self.y_dtype, self.mod_dtype} <= {bf16, f32}:
            raise ValueError("types are bfloat16 or float32")
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.shape = AdalnShape.make(B, T_txt, T_img, C, norm, post or "none", self.x_dtype == f32, self.y_dtype == f32,
                                     self.mod_dtype == f32, eps, alpha)
        self._ws_bytes = rlk_adaln_workspace_bytes(self.shape)
        if self._ws_bytes == 0:
            raise RlkError(1, "AdaLN: invalid shape")
        self._f32, self._index = f32, -1 if self.device.index is None else self.device.index
        # expected sizes of each stream's tensors, None where it has no tokens
        live = (T_txt > 0, T_img > 0)
        self._live = live
        self._rows = tuple(torch.Size((B, T, C)) if T else None for T in (T_txt, T_img))
        self._stats = tuple(torch.Size((B, T, 2)) if T else None for T in (T_txt, T_img))
        self._sums = tuple(torch.Size((B, C)) if on else None for on in live)
        self._vector = tuple(torch.Size((C,)) if on else None for on in live)
        # sizes and type of each output
        x, y, f = self.x_dtype, self.y_dtype, self._f32
        self._kinds = {"y": (self._rows, y), "r": (self._rows, x), "stats": (self._stats, f), "post_stats": (self._stats, f),
                       "dx": (self._rows, x), "dh": (self._rows, y), "dgate": (self._sums, f), "dscale": (self._sums, f),
                       "dshift": (self._sums, f), "dw": (self._vector, f), "dw_post": (self._vector, f)}
        self._shapes = {}  # the call's shape struct by the modulation's sample stride
        self.workspace, self._streams = None, set()  # of the backward, allocated at its first call; used by

    # ---- checks
    def _weights(self, name, pair):
        """Pointers of a pair of optional [C] weights."""
        if pair is None or (pair[0] is None and pair[1] is None):
            return _NONE
        for i in (0, 1):
            if pair[i] is not None and self._vector[i] is None:
                self._bad(name, i, pair[i], None, None)
        return self._need(name, pair, self._f32, tuple(None if t is None else w for t, w in zip(pair, self._vector)))

    def _view(self, name, i, t, strides):
        """Pointer of a stream's [B, C] modulation view; its sample stride goes to `strides`."""
        if t is None:
            return None
        want = self._sums[i]
        s = t.stride()
        if want is None or t.dtype is not self.mod_dtype or t.shape != want or s[1] != 1 or t.get_device() != self._index:
            sh = self.shape
            raise ValueError(f"{name}[{i}] must be a {self.mod_dtype} [{sh.B}, {sh.C}] view with unit column stride on "
                             f"{self.device} (None without tokens), got {t.dtype} {tuple(t.shape)} on {t.device}")
        strides.append(s[0])
        return t.data_ptr()

    def _mods(self, *named):
        """The call's shape (with the views' sample stride) and the pointers of pairs of [B, C] views."""
        strides, res = [], []
        for name, pair in named:
            if pair is None:
                res.append(_NONE)
                continue
            if len(pair) != 2:
                raise ValueError(f"{name} must be a (text, image) pair")
            res.append((self._view(name, 0, pair[0], strides), self._view(name, 1, pair[1], strides)))
        stride = self.shape.C
        if strides and self.shape.B > 1:  # (a single sample's stride says nothing)
            stride = strides[0]
            if strides.count(stride) != len(strides):
                raise ValueError(f"scale, shift and gate must have one sample stride, got {sorted(set(strides))}")
            if stride < self.shape.C:
                raise ValueError(f"scale, shift and gate need rows of their own for every sample, got the stride {stride}")
        call = self._shapes.get(stride)
        if call is None:
            call = AdalnShape.from_buffer_copy(self.shape)
            call.mod_stride = stride
            self._shapes[stride] = call
        return call, res

    def _structs(self, cls, *pairs):
        """One struct of pointers per stream, its fields in order (None for a stream without tokens)."""
        return [cls(*[p[i] for p in pairs]) if self._live[i] else None for i in (0, 1)]

    # ---- calls
    def modulation(self, x, scale, shift, w=None, out=None, stream=None):
        """y = hat(x) * w * (1 + scale) + shift. Returns y and stats."""
        px = self._need("x", x, self.x_dtype, self._rows)
        call, (pscale, pshift) = self._mods(("scale", scale), ("shift", shift))
        pw = self._weights("w", w)
        out, p = self._outputs(out, ("y", "stats"), stream)
        _require_current(self.device)
        io = self._structs(AdalnIo, px, _NONE, _NONE, pscale, pshift, pw, _NONE, _NONE, p["y"], p["stats"])
        rlk_adaln_modulation_fwd(call, io, _raw_stream(stream, self._index))
        return out

    def gate_residual(self, x, h, gate, scale, shift, w=None, w_post=None, want_y=True, out=None, stream=None):
        """r = x + alpha * gate * u (u = h, or hat(h) * w_post with a norm
        after the sublayer), y = modulation of r. Returns r, and with want_y y
        and stats, and with a norm after the sublayer post_stats. ``out`` may
        hold x itself as r."""
        px = self._need("x", x, self.x_dtype, self._rows)
        ph = self._need("h", h, self.y_dtype, self._rows)
        call, (pgate, pscale, pshift) = self._mods(("gate", gate), ("scale", scale), ("shift", shift))
        pw, pwp = self._weights("w", w), self._weights("w_post", w_post)
        want = ("r", "y", "stats") if want_y else ("r",)
        if call.post:
            want += ("post_stats",)
        out, p = self._outputs(out, want, stream)
        _require_current(self.device)
        io = self._structs(AdalnIo, px, ph, pgate, pscale, pshift, pw, pwp, p["r"], p.get("y", _NONE),
                           p.get("stats", _NONE), p.get("post_stats", _NONE))
        rlk_adaln_gate_residual_fwd(call, io, _raw_stream(stream, self._index))
        return out

    def modulation_bwd(self, x, scale, stats, dy, dr=None, w=None, out=None, stream=None):
        """Gradients of the modulation: dx (with dr, the gradient that reaches
        x by the residual path, added), dscale and dshift [B, C] and, with w,
        dw [C], all sums float32. ``out`` may hold dr itself as dx."""
        px = self._need("x", x, self.x_dtype, self._rows)
        pst = self._need("stats", stats, self._f32, self._stats)
        pdy = self._need("dy", dy, self.y_dtype, self._rows)
        pdr = _NONE if dr is None else self._need("dr", dr, self.x_dtype, self._rows)
        call, (pscale,) = self._mods(("scale", scale))
        pw = self._weights("w", w)
        want = ("dx", "dscale", "dshift") if pw is _NONE else ("dx", "dscale", "dshift", "dw")
        out, p = self._outputs(out, want, stream)
        _require_current(self.device)
        io = self._structs(AdalnIo, px, _NONE, _NONE, pscale, _NONE, pw, _NONE, _NONE, _NONE, pst)
        grad = self._structs(AdalnGrad, pdy, pdr, p["dx"], _NONE, _NONE, p["dscale"], p["dshift"], p.get("dw", _NONE))
        handle = _raw_stream(stream, self._index)
        rlk_adaln_modulation_bwd(call, io, grad, _workspace(self, self._ws_bytes, stream, handle), None, handle)
        return out

    def gate_residual_bwd(self, r, h, gate, scale, stats, dy, dr=None, w=None, w_post=None, post_stats=None, out=None,
                          stream=None):
        """Gradients of gate_residual from r and the statistics it left: dx,
        dh, dgate, with dy (None: y was not used) dscale and dshift, with w
        dw, with w_post dw_post. dr is the gradient that reaches r by the
        residual path. ``out`` may hold dr itself as dx."""
        f32, rows = self._f32, self._rows
        pr = self._need("r", r, self.x_dtype, rows)
        ph = self._need("h", h, self.y_dtype, rows)
        if dy is None and dr is None:
            raise ValueError("dy and dr cannot both be None")
        pdr = _NONE if dr is None else self._need("dr", dr, self.x_dtype, rows)
        call, (pgate, pscale) = self._mods(("gate", gate), ("scale", scale))
        pw, pwp = self._weights("w", w), self._weights("w_post", w_post)
        want = ("dx", "dh", "dgate")
        pdy = pst = pps = _NONE
        if dy is not None:
            pdy = self._need("dy", dy, self.y_dtype, rows)
            pst = self._need("stats", stats, f32, self._stats)
            want += ("dscale", "dshift") if pw is _NONE else ("dscale", "dshift", "dw")
        if call.post:
            pps = self._need("post_stats", post_stats, f32, self._stats)
            if pwp is not _NONE:
                want += ("dw_post",)
        out, p = self._outputs(out, want, stream)
        _require_current(self.device)
        io = self._structs(AdalnIo, _NONE, ph, pgate, pscale, _NONE, pw, pwp, pr, _NONE, pst, pps)
        grad = self._structs(AdalnGrad, pdy, pdr, p["dx"], p["dh"], p["dgate"], p.get("dscale", _NONE),
                             p.get("dshift", _NONE), p.get("dw", _NONE), p.get("dw_post", _NONE))
        handle = _raw_stream(stream, self._index)
        rlk_adaln_gate_residual_bwd(call, io, grad, _workspace(self, self._ws_bytes, stream, handle), None, handle)
        return out


class AdamW:
    """AdamW over a list of parameters (see rlk_adamw_step in the header).

    ``params`` are contiguous CUDA tensors, float32, or bfloat16 with a float32
    master copy (taken from ``masters``, or made from the parameter). States
    are zero unless given: ``m`` and ``v`` float32 (state_bits 32) or
    float8_e4m3fn with uint8 ``m_scale`` and ``v_scale`` per 32 elements
    (state_bits 8). ``weight_decay`` and ``lr_scale`` are one number or one per
    parameter. ``keys`` (default 0, 1, ...) name the parameters to the 8-bit
    states' rounding. ``grads``, bfloat16 or float32, may be held here (buffers
    that a backward pass writes anew for every step) or given to each call.
    ``params``, ``masters``, ``m``, ``v``, ``m_scale`` and ``v_scale`` hold the
    tensors in use, one entry a parameter: what a checkpoint keeps, and what the
    constructor takes to go on from one. They stay the same tensors for the
    object's life, those of the masters and states its own over the memory of the
    ones given: load values into them with ``copy_``. The calls refuse a list
    with a tensor whose ``data`` was replaced since (by whoever holds it: the
    parameters, the gradients, and what was read from the other lists), and its
    old memory stays allocated. ``lr`` may be set at any time. grad_norm's
    calls share one workspace: calls that may overlap on the GPU need an object
    each. An object outlives the graphs that captured its calls, and its calls on
    a stream that is given as an address. States and masters that are made here
    are written on the current stream."""

    def __init__(self, params, masters=None, state_bits: int = 32, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay=0.01, lr_scale=1.0, seed: int = 0, keys=None, grads=None, m=None, v=None, m_scale=None,
                 v_scale=None):
        import torch
        f32, bf16 = torch.float32, torch.bfloat16
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        n = len(params)
        if n == 0:
            raise ValueError("no parameters given")
        self._params, self.state_bits, self.lr = tuple(params), state_bits, float(lr)
        self.device = self.params[0].device
        self._index = self.device.index
        each = lambda x: list(x) if isinstance(x, (list, tuple)) else [x] * n  # noqa: E731
        decay, share, keys = each(weight_decay), each(lr_scale), list(range(n)) if keys is None else list(keys)
        masters = [None] * n if masters is None else list(masters)
        code = torch.float8_e4m3fn if state_bits == 8 else f32
        blocks = [-(-p.numel() // 32) for p in self.params]

        def states(given, dtype, sizes):
            if given is None:
                return tuple(torch.zeros(k, dtype=dtype, device=self.device) for k in sizes)
            return tuple(given)
        sizes = [p.numel() for p in self.params]
        m, v = states(m, code, sizes), states(v, code, sizes)
        m_scale = states(m_scale, torch.uint8, blocks) if state_bits == 8 else (None,) * n
        v_scale = states(v_scale, torch.uint8, blocks) if state_bits == 8 else (None,) * n
        if not len(decay) == len(share) == len(keys) == len(masters) == len(m) == len(v) == len(m_scale) == len(v_scale) == n:
            raise ValueError(f"expected one entry for each of the {n} parameters")
        if not all(0 <= int(k) < 2 ** 32 for k in [seed, *keys]):
            raise ValueError("seed and keys must be in 0 .. 2^32 - 1")
        self._list = (AdamwTensor * n)()
        for i, p in enumerate(self.params):
            if p.dtype not in (f32, bf16):
                raise ValueError(f"parameter {i} must be float32 or bfloat16, got {p.dtype}")
            if p.dtype == f32 and masters[i] is not None:
                raise ValueError(f"parameter {i} is float32 and takes no master")
            if p.dtype == bf16 and masters[i] is None:
                masters[i] = p.detach().float().contiguous()
            for name, t, dtype, k in (("parameter", p, p.dtype, sizes[i]), ("master", masters[i], f32, sizes[i]),
                                      ("m", m[i], code, sizes[i]), ("v", v[i], code, sizes[i]),
                                      ("m_scale", m_scale[i], torch.uint8, blocks[i]),
                                      ("v_scale", v_scale[i], torch.uint8, blocks[i])):
                if t is not None:
                    self._dense(f"{name} {i}", t, (dtype,), k)
            e = self._list[i]
            e.p, e.master, e.m, e.v = _ptr(p), _ptr(masters[i]), _ptr(m[i]), _ptr(v[i])
            e.m_scale, e.v_scale, e.n = _ptr(m_scale[i]), _ptr(v_scale[i]), sizes[i]
            e.lr_scale, e.weight_decay, e.state_bits, e.key = float(share[i]), float(decay[i]), state_bits, int(keys[i])
        self._lists = {"masters": tuple(masters), "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale}
        # The call's list holds addresses. The storages behind them are held here, so that they stay allocated, and
        # the tensors that someone else holds too are looked at for still being over them: parameters and gradients,
        # and a list of states once it was read (180 tensors with 8-bit states and masters are 1200 addresses, 70 us a
        # call; parameters and gradients are 21).
        self._storages = {name: [None if t is None else t.untyped_storage() for t in held]
                          for name, held in [("params", self._params), *self._lists.items()]}
        self._data_ptr = torch.Tensor.data_ptr
        self._params_at = list(map(self._data_ptr, self._params))
        self._handed, self._others, self._others_at = set(), [], []
        self._grads = None
        if grads is not None:
            self._take(grads)
        self._args = AdamwArgs(lr=self.lr, beta1=float(betas[0]), beta2=float(betas[1]), eps=float(eps), seed=int(seed))
        self._args_ref = ctypes.byref(self._args)
        self.workspace, self._streams = None, set()  # of grad_norm, allocated at its first call; used by

    def _hand_out(self, name):
        """One of the lists, for someone to read: tensors of the object's own, looked at from now on."""
        if name not in self._handed:
            import torch
            held, field = [], "master" if name == "masters" else name
            for t, storage, e in zip(self._lists[name], self._storages[name], self._list):
                if t is not None:
                    at = getattr(e, field) or 0
                    if t.data_ptr() == at:
                        t = t.detach()
                    else:  # whoever gave it has replaced its data
                        n = t.element_size()
                        size = -(-e.n // 32) if field.endswith("scale") else e.n
                        t = torch.empty(0, dtype=t.dtype, device=self.device).set_(storage, (at - storage.data_ptr()) // n, (size,))
                    self._others.append(t)
                    self._others_at.append(at)
                held.append(t)
            self._lists[name] = tuple(held)
            self._handed.add(name)
        return self._lists[name]

    params = property(lambda self: self._params)
    grads = property(lambda self: self._grads)
    masters = property(lambda self: self._hand_out("masters"))
    m = property(lambda self: self._hand_out("m"))
    v = property(lambda self: self._hand_out("v"))
    m_scale = property(lambda self: self._hand_out("m_scale"))
    v_scale = property(lambda self: self._hand_out("v_scale"))

    def _same(self, tensors, addresses):
        if list(map(self._data_ptr, tensors)) != addresses:
            raise ValueError("a tensor's data was replaced: copy_ into it, or make a new object (gradients: give them anew)")

    def _dense(self, name, t, dtypes, n):
        if t.dtype not in dtypes or t.numel() != n or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"{name} must be a contiguous tensor of {n} elements ({dtypes}) on {self.device}, got "
                             f"{t.dtype} {tuple(t.shape)} on {t.device}")

    def _take(self, grads):
        """The list's gradient buffers from now on."""
        import torch
        grads = tuple(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"expected {len(self.params)} gradients, got {len(grads)}")
        f32, types, device = torch.float32, (torch.float32, torch.bfloat16), self.device
        for i, (g, p, e) in enumerate(zip(grads, self.params, self._list)):
            if g.dtype not in types or g.numel() != e.n or not g.is_contiguous() or g.device != device:
                self._dense(f"gradient {i}", g, types, e.n)
            if g.dim() != 1 and g.shape != p.shape:
                raise ValueError(f"gradient {i} must be {tuple(p.shape)} or flat, got {tuple(g.shape)}")
        self._grads_at = list(map(self._data_ptr, grads))
        for e, g, at in zip(self._list, grads, self._grads_at):
            e.g, e.g_dtype = at, int(g.dtype is f32)
        self._grads, self._grad_storages = grads, list(map(torch.Tensor.untyped_storage, grads))

    def _ready(self, grads):
        if grads is not None:
            self._take(grads)
        if self._grads is None:
            raise ValueError("no gradients given")
        self._same(self._grads, self._grads_at)
        _require_current(self.device)

    def _scalar(self, name, t, dtype):
        if t is None:
            return None
        if t.dtype != dtype or t.numel() != 1 or t.device != self.device:
            raise ValueError(f"{name} must be one {dtype} value on {self.device}")
        return t.data_ptr()

    def grad_norm(self, max_norm: float = float("inf"), pre_scale: float = 1.0, grads=None, out=None, stream=None):
        """float32 [2] on the device: the gradients' global norm (times
        pre_scale) and the factor (pre_scale included) that clips it to
        max_norm, NaN if the norm is not finite."""
        import torch
        self._ready(grads)
        n = len(self._params)
        if out is None:
            out = _empty(2, torch.float32, self.device, stream)
        else:
            self._dense("out", out, (torch.float32,), 2)
        handle = _raw_stream(stream, self._index)
        ws = self.workspace
        if ws is None or handle not in self._streams:
            ws = _workspace(self, rlk_grad_norm_workspace_bytes(self._list, n), stream, handle)
        rc = lib().rlk_grad_norm(self._list, n, float(pre_scale), float(max_norm), out.data_ptr(), ws.data_ptr(), ws.numel(),
                                 handle)
        if rc:
            _check(rc, "rlk_grad_norm")
        return out

    def step(self, step, lr=None, grad_scale=None, grads=None, stream=None):
        """One update, in place. ``step`` is this step's number from 1 on, and
        ``lr`` the rate if not the constructor's; each an ordinary number, or a
        device tensor of one value (int64, float32) that is read when the
        kernels run, as a captured step needs. ``grad_scale`` is one float32
        value on the device, such as grad_norm(...)[1:]. If it is not finite, or
        a device ``step`` is not in 1 .. 2^31 - 1, nothing is changed."""
        import torch
        self._same(self._params, self._params_at)
        if self._others:
            self._same(self._others, self._others_at)
        self._ready(grads)
        a = self._args
        a.step_dev = a.lr_dev = None
        if isinstance(step, torch.Tensor):
            a.step_dev, a.step = self._scalar("step", step, torch.int64), 1
        else:
            a.step = int(step)
        if isinstance(lr, torch.Tensor):
            a.lr_dev, a.lr = self._scalar("lr", lr, torch.float32), 0.0
        else:
            a.lr = self.lr if lr is None else float(lr)
        a.grad_scale = self._scalar("grad_scale", grad_scale, torch.float32)
        rc = lib().rlk_adamw_step(self._list, len(self._params), self._args_ref, _raw_stream(stream, self._index))
        if rc:
            _check(rc, "rlk_adamw_step")


def _cuda_device(device):
    import torch
    device = torch.device(device)
    if device.type == "cuda" and device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return device


_GRADS = ("dx", "dw", "db")


class Fp8Projection(_Pairs):
    """Buffers + calls of one projection y = x W^T + b of both streams in 8-bit floating point (rlk_fp8_quantize,
    rlk_fp8_gemm), each stream with weights of its own.

    x and dx are (text, image) pairs, bf16 [B, T_txt, n_in] and [B, T_img, n_in], y and dy likewise with n_out; a pair's
    text is None if T_txt is 0 and its image None if T_img is 0. ``set_weights`` rounds the weights to codes that the
    object holds until the next call of it. Values are rounded to e4m3 with a power-of-two scale for each 128 of them,
    gradients to ``grad_format`` (e4m3 or e5m2). n_in and n_out are multiples of 8.

    Every call returns its outputs as a dict of pairs; passing that dict back as ``out`` reuses its buffers. The calls
    share one workspace and the weights' codes: calls that may overlap on the GPU (other streams, graphs replayed at
    the same time) need an object each. An object outlives the graphs that captured its calls, and its calls on a stream
    that is given as an address."""

    def __init__(self, B: int, T_txt: int, T_img: int, n_in: int, n_out: int, out_dtype=None, dw_dtype=None,
                 grad_format: str = "e4m3", device="cuda"):
        import torch
        bf16, f32 = torch.bfloat16, torch.float32
        self.out_dtype, self.dw_dtype = out_dtype or bf16, dw_dtype or f32
        if not {self.out_dtype, self.dw_dtype} <= {bf16, f32}:
            raise ValueError("types are bfloat16 or float32")
        if grad_format not in FP8_FORMATS:
            raise ValueError(f"grad_format must be one of {sorted(FP8_FORMATS)}")
        if B < 1 or T_txt < 0 or T_img < 0 or T_txt + T_img == 0 or not all(
                8 <= k <= 1 << 20 and k % 8 == 0 for k in (n_in, n_out)) or B * max(T_txt, T_img) >= (1 << 31) - 256:
            raise RlkError(1, "Fp8Projection: invalid shape")
        self.device = _cuda_device(device)
        self._index = -1 if self.device.index is None else self.device.index
        self.B, self.T, self.n_in, self.n_out = B, (T_txt, T_img), n_in, n_out
        self._grad = FP8_FORMATS[grad_format]
        self._live = [i for i in (0, 1) if self.T[i] > 0]
        self._tokens = tuple(B * t for t in self.T)
        on = lambda make: tuple(torch.Size(make(t)) if t else None for t in self.T)  # noqa: E731
        rows, srows = rlk_fp8_row_bytes, rlk_fp8_scale_row_bytes
        code, byte = torch.float8_e4m3fn, torch.uint8
        self._x = on(lambda t: (B, t, n_in))
        self._y = on(lambda t: (B, t, n_out))
        self._w = on(lambda t: (n_out, n_in))
        self._b = on(lambda t: (n_out,))
        self._kinds = {"y": (self._y, self.out_dtype), "dx": (self._x, bf16), "dw": (self._w, self.dw_dtype),
                       "db": (self._b, f32), "xt": (on(lambda t: (n_in, rows(B * t))), code),
                       "xt_scale": (on(lambda t: (n_in, srows(B * t))), byte)}
        # weights as they are and turned, their scales
        sizes = ((n_out, rows(n_in)), (n_out, srows(n_in)), (n_in, rows(n_out)), (n_in, srows(n_out)))
        self._codes = [None if not t else tuple(torch.empty(k, dtype=byte, device=self.device) for k in sizes) for t in self.T]
        self._at = [None if c is None else tuple(k.data_ptr() for k in c) for c in self._codes]
        self._set = False
        # the workspace: codes and scales of x, or of dy as it is and turned and the sums of its columns
        self._fwd, self._bwd, fwd, bwd = {}, {}, 0, 0

        def place(at, sizes):
            starts = []
            for k in sizes:
                starts.append(at)
                at += -(-k // 256) * 256
            return at, starts
        for i in self._live:
            t = self._tokens[i]
            fwd, self._fwd[i] = place(fwd, (t * rows(n_in), t * srows(n_in)))
            bwd, self._bwd[i] = place(bwd, (t * rows(n_out), t * srows(n_out), n_out * rows(t), n_out * srows(t),
                                            rlk_fp8_quant_workspace_bytes(t, n_out)))
        self._ws_bytes = max(fwd, bwd)
        self._weight_call = (Fp8Quant * len(self._live))(*[
            Fp8Quant(None, *self._at[i], None, None, n_out, n_in, n_in, 0, 0, 1, 0) for i in self._live])
        self._calls = {}  # the C calls' arguments by kind of call, once there is a workspace
        self.workspace, self._streams = None, set()

    def set_weights(self, w, stream=None) -> None:
        """Rounds a pair of weights, float32 or bfloat16 [n_out, n_in], to codes in blocks of 128 x 128."""
        import torch
        dtype = next((t.dtype for t in w if t is not None), None)
        if dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("weights are bfloat16 or float32")
        pw = self._need("w", w, dtype, self._w)
        _require_current(self.device)
        handle = _raw_stream(stream, self._index)
        if handle not in self._streams:
            self._record(stream, handle)
        items = self._weight_call
        for e, i in zip(items, self._live):
            e.x, e.x_dtype = pw[i], int(dtype is torch.float32)
        self._run(items, None, handle)
        self._set = True

    def _record(self, stream, handle):
        """The weights' codes wait for every torch stream that uses them when the object goes."""
        import torch
        s = torch.cuda.current_stream(self.device) if stream is None else stream
        if not isinstance(s, int):
            for c in self._codes:
                for t in c or ():
                    t.record_stream(s)

    def _ready(self, stream):
        if not self._set:
            raise ValueError("no weights given: set_weights comes first")
        _require_current(self.device)
        handle = _raw_stream(stream, self._index)
        if handle not in self._streams:  # (those have a workspace)
            self._record(stream, handle)
            _workspace(self, self._ws_bytes, stream, handle)
        return handle

    def _out(self, out, names, stream):
        """The outputs of these names and their pointers (new ones without what a reuse is checked by: that takes
        longer than the smallest kernels, and most calls' outputs are not passed back)."""
        if out is not None:
            return self._outputs(out, names, stream)
        device, kinds, out, p = self.device, self._kinds, {}, {}
        for k in names:
            (t, i), dtype = kinds[k]
            t = None if t is None else _empty(t, dtype, device, stream)
            i = None if i is None else _empty(i, dtype, device, stream)
            out[k], p[k] = (t, i), (None if t is None else t.data_ptr(), None if i is None else i.data_ptr())
        return out, p

    def _vectors(self, name, pair, dtype, sizes):
        if pair is None:
            return _NONE
        if len(pair) != 2:
            raise ValueError(f"{name} must be a (text, image) pair")
        t, i = pair
        return self._need(name, pair, dtype, (None if t is None else sizes[0], None if i is None else sizes[1]))

    def forward(self, x, bias=None, train: bool = False, out=None, stream=None):
        """y, and with train what the backward needs of x: xt and xt_scale, its codes turned. bias is a pair of bf16
        [n_out], either of them or both None (0)."""
        import torch
        bf16 = torch.bfloat16
        px = self._need("x", x, bf16, self._x)
        pb = self._vectors("bias", bias, bf16, self._b)
        out, p = self._out(out, ("y", "xt", "xt_scale") if train else ("y",), stream)
        handle = self._ready(stream)
        quant, product = self._calls.get(train) or self._fwd_calls(train, self.workspace.data_ptr())
        py, xt, xs = p["y"], p.get("xt"), p.get("xt_scale")
        for n, i in enumerate(self._live):  # (the rest of a call stays what it is)
            f = product[n]
            f.bias, f.d = pb[i], py[i]
            if quant is None:
                f.a = px[i]
                continue
            e = quant[n]
            e.x = px[i]
            if train:
                e.qt, e.qt_scale = xt[i], xs[i]
        self._run(quant, product, handle)
        return out

    def _fwd_calls(self, train, ws):
        n_in, n_out, bf16 = self.n_in, self.n_out, self.out_dtype.itemsize == 2
        quant, product = [], []
        if not train and max(self._tokens) <= FP8_FEW_ROWS and n_in <= FP8_FEW_K:  # a few tokens: rounded by the product
            for i in self._live:
                t, w = self._tokens[i], self._at[i]
                product.append(Fp8Product(None, None, w[0], w[1], None, None, t, n_out, n_in, n_out, 0, 0, 0 if bf16 else 1, 0, 1, 0))
            self._calls[train] = None, (Fp8Product * len(product))(*product)
            return self._calls[train]
        for i in self._live:
            q, s, t, w = ws + self._fwd[i][0], ws + self._fwd[i][1], self._tokens[i], self._at[i]
            quant.append(Fp8Quant(None, q, s, None, None, None, None, t, n_in, n_in, 0, 0, 0, 0))
            product.append(Fp8Product(q, s, w[0], w[1], None, None, t, n_out, n_in, n_out, 0, 0, 0 if bf16 else 1, 0))
        self._calls[train] = (Fp8Quant * len(quant))(*quant), (Fp8Product * len(product))(*product)
        return self._calls[train]

    def _run(self, quant, product, handle):
        if quant is not None:
            rc = lib().rlk_fp8_quantize(quant, len(quant), handle)
            if rc:
                _check(rc, "rlk_fp8_quantize")
        if product is not None:
            rc = lib().rlk_fp8_gemm(product, len(product), handle)
            if rc:
                _check(rc, "rlk_fp8_gemm")

    def backward(self, dy, saved, want=("dx", "dw", "db"), accumulate: bool = False, out=None, stream=None):
        """Gradients named in ``want``: dx (bf16), dw (float32 or the constructor's dw_dtype), db (float32). ``saved`` is
        what forward(train=True) returned (dw only; else None may be given). With accumulate, dw is added to the one in
        ``out`` (float32)."""
        import torch
        bf16, f32 = torch.bfloat16, torch.float32
        if want != _GRADS:
            want = tuple(k for k in _GRADS if k in want)
            if not want:
                raise ValueError("want must name dx, dw or db")
        pdy = self._need("dy", dy, bf16, self._y)
        pxt = pxs = _NONE
        if "dw" in want:
            if saved is None or "xt" not in saved:
                raise ValueError("dw needs what forward(train=True) returned")
            (sizes, dtype), (scale_sizes, scale_dtype) = self._kinds["xt"], self._kinds["xt_scale"]
            pxt = self._need("xt", saved["xt"], dtype, sizes)
            pxs = self._need("xt_scale", saved["xt_scale"], scale_dtype, scale_sizes)
        if accumulate and ("dw" not in want or out is None or self.dw_dtype is not f32):
            raise ValueError("accumulate needs out with a float32 dw")
        out, p = self._out(out, want, stream)
        handle = self._ready(stream)
        dx, dw, db = ("dx" in want), ("dw" in want), ("db" in want)
        quant, product = self._calls.get(want) or self._bwd_calls(want, self.workspace.data_ptr())
        k = 0
        for n, i in enumerate(self._live):
            quant[n].x = pdy[i]
            if db:
                quant[n].col_sum = p["db"][i]
            if dx:
                product[k].d = p["dx"][i]
                k += 1
            if dw:
                e = product[k]
                e.b, e.b_scale, e.d, e.accumulate = pxt[i], pxs[i], p["dw"][i], int(accumulate)
                k += 1
        self._run(quant, product, handle)
        return out

    def _bwd_calls(self, want, ws):
        n_in, n_out, f, f32 = self.n_in, self.n_out, self._grad, self.dw_dtype.itemsize == 4
        dx, dw, db = ("dx" in want), ("dw" in want), ("db" in want)
        quant, product = [], []
        for i in self._live:
            q, s, qt, st, part = [ws + k for k in self._bwd[i]]
            t, w = self._tokens[i], self._at[i]
            turned = dw or not dx  # (db alone: the sums come with one of the two)
            quant.append(Fp8Quant(None, q if dx else None, s if dx else None, qt if turned else None, st if turned else None,
                                  None, part if db else None, t, n_out, n_out, 0, f, 0, 0))
            if dx:
                product.append(Fp8Product(q, s, w[2], w[3], None, None, t, n_in, n_out, n_in, f, 0, 0, 0))
            if dw:
                product.append(Fp8Product(qt, st, None, None, None, None, n_out, n_in, t, n_in, f, 0, int(f32), 0))
        self._calls[want] = (Fp8Quant * len(quant))(*quant), (Fp8Product * len(product))(*product) if product else None
        return self._calls[want]


POLYNOMIAL = (3.4445, -4.7750, 2.0315)


def _matrix(name, t, dtypes, device, shape=None):
    if t.dim() != 2 or t.dtype not in dtypes or (shape is not None and t.shape != shape) or not t.is_contiguous() or \
            t.device != device:
        want = "2-D" if shape is None else tuple(shape)
        raise ValueError(f"{name} must be a contiguous {want} tensor ({dtypes}) on {device}, got {t.dtype} {tuple(t.shape)} on "
                         f"{t.device}")


def orthogonalize(matrices, out=None, iterations: int = 5, coefficients=POLYNOMIAL, eps: float = 1e-7, stream=None):
    """Newton-Schulz products X = a X + (b A + c A A) X, A = X X^T, on each of a list of matrices (bf16 or float32 on one
    device, of any sizes), from X = x / (||x||_F + eps) on: singular values go towards 1. Returns bf16 matrices, those of
    ``out`` if it is given. See rlk_orthogonalize in the header."""
    import torch
    bf16, f32 = torch.bfloat16, torch.float32
    matrices = list(matrices)
    if not matrices:
        return []
    device = matrices[0].device
    for i, x in enumerate(matrices):
        _matrix(f"matrix {i}", x, (bf16, f32), device)
    _require_current(device)
    if out is None:
        out = [_empty(x.shape, bf16, device, stream) for x in matrices]
    if len(out) != len(matrices):
        raise ValueError(f"expected {len(matrices)} outputs, got {len(out)}")
    for i, (x, o) in enumerate(zip(matrices, out)):
        _matrix(f"output {i}", o, (bf16,), device, x.shape)
    n = len(matrices)
    a, b, c = (float(k) for k in coefficients)
    items = (MuonMatrix * n)(*[MuonMatrix(o.data_ptr() or None, None, x.data_ptr() or None, None, x.shape[0], x.shape[1], 0.0, 0.0,
                                          int(x.dtype is f32), 0) for x, o in zip(matrices, out)])
    args = MuonArgs(a=a, b=b, c=c, eps=float(eps), iterations=int(iterations))
    size = rlk_muon_workspace_bytes(items)
    if size == 0:
        raise RlkError(1, "orthogonalize: invalid sizes")
    rlk_orthogonalize(items, args, _empty(size, torch.uint8, device, stream), _raw_stream(stream, device.index))
    return out


class Muon:
    """Muon over a list of matrices (see rlk_muon_step in the header), for the projections' weights; vectors and gains go
    to AdamW.

    ``params`` are contiguous 2-D CUDA tensors, float32, or bfloat16 with a float32 master copy (taken from ``masters``,
    or made from the parameter). The momentum ``m`` is float32 of the parameter's shape, zero unless given.
    ``weight_decay`` and ``lr_scale`` are one number or one per parameter. An update has the root mean square lr *
    update_rms (at full rank), so that AdamW's rates serve here too. ``grads``, bfloat16 or float32, may be held here or
    given to each call. ``params``, ``masters`` and ``m`` hold the tensors in use: load values into them with ``copy_``. A
    call refuses a list with a tensor whose ``data`` was replaced. ``lr`` may be set at any time. The calls share one
    workspace: calls that may overlap on the GPU need an object each. An object outlives the graphs that captured its
    calls, and its calls on a stream that is given as an address. What is made here is written on the current stream."""

    def __init__(self, params, masters=None, lr: float = 1e-3, momentum: float = 0.95, nesterov: bool = True, weight_decay=0.01,
                 lr_scale=1.0, update_rms: float = 0.2, iterations: int = 5, coefficients=POLYNOMIAL, eps: float = 1e-7,
                 grads=None, m=None):
        import torch
        f32, bf16 = torch.float32, torch.bfloat16
        n = len(params)
        if n == 0:
            raise ValueError("no parameters given")
        self.params, self.lr = tuple(params), float(lr)
        self.device = self.params[0].device
        self._index = self.device.index
        each = lambda x: list(x) if isinstance(x, (list, tuple)) else [x] * n  # noqa: E731
        decay, share = each(weight_decay), each(lr_scale)
        masters = [None] * n if masters is None else list(masters)
        m = [None] * n if m is None else list(m)
        if not len(decay) == len(share) == len(masters) == len(m) == n:
            raise ValueError(f"expected one entry for each of the {n} parameters")
        self._list = (MuonMatrix * n)()
        for i, p in enumerate(self.params):
            _matrix(f"parameter {i}", p, (f32, bf16), self.device)
            if p.dtype == f32 and masters[i] is not None:
                raise ValueError(f"parameter {i} is float32 and takes no master")
            if p.dtype == bf16 and masters[i] is None:
                masters[i] = p.detach().float()
            if m[i] is None:
                m[i] = torch.zeros(p.shape, dtype=f32, device=self.device)
            if masters[i] is not None:
                _matrix(f"master {i}", masters[i], (f32,), self.device, p.shape)
            _matrix(f"m {i}", m[i], (f32,), self.device, p.shape)
            e = self._list[i]
            e.p, e.master, e.m = (None if t is None else t.data_ptr() or None for t in (p, masters[i], m[i]))
            e.rows, e.cols, e.lr_scale, e.weight_decay = p.shape[0], p.shape[1], float(share[i]), float(decay[i])
        self.masters, self.m = tuple(masters), tuple(m)
        self._held = [t for t in (*self.params, *self.masters, *self.m) if t is not None]
        self._held_at = [t.data_ptr() for t in self._held]
        # (the list holds addresses: the storages behind them stay allocated)
        self._storages = [t.untyped_storage() for t in self._held]
        a, b, c = (float(k) for k in coefficients)
        self._args = MuonArgs(lr=self.lr, momentum=float(momentum), update_rms=float(update_rms), a=a, b=b, c=c, eps=float(eps),
                              iterations=int(iterations), nesterov=int(bool(nesterov)))
        self.grads = None
        if grads is not None:
            self._take(grads)
        self._ws_bytes = rlk_muon_workspace_bytes(self._list)
        if self._ws_bytes == 0:
            raise RlkError(1, "Muon: invalid sizes")
        self.workspace, self._streams = None, set()

    def _take(self, grads):
        import torch
        grads = tuple(grads)
        if len(grads) != len(self.params):
            raise ValueError(f"expected {len(self.params)} gradients, got {len(grads)}")
        for i, (g, p) in enumerate(zip(grads, self.params)):
            _matrix(f"gradient {i}", g, (torch.float32, torch.bfloat16), self.device, p.shape)
        self._grads_at = [g.data_ptr() for g in grads]
        for e, g, at in zip(self._list, grads, self._grads_at):
            e.g, e.g_dtype = at or None, int(g.dtype is torch.float32)
        self.grads, self._grad_storages = grads, [g.untyped_storage() for g in grads]

    def step(self, lr=None, grad_scale=None, grads=None, stream=None):
        """One update, in place. ``lr`` is the rate if not the constructor's, a number, or a float32 device tensor of one
        value that is read when the kernels run, as a captured step needs, and gives the bytes of the same number.
        ``grad_scale`` is one float32 value on the device, such as AdamW.grad_norm(...)[1:]; if it is not finite, nothing
        is changed."""
        import torch
        if grads is not None:
            self._take(grads)
        if self.grads is None:
            raise ValueError("no gradients given")
        if [t.data_ptr() for t in self._held] != self._held_at or [t.data_ptr() for t in self.grads] != self._grads_at:
            raise ValueError("a tensor's data was replaced: copy_ into it, or make a new object (gradients: give them anew)")
        _require_current(self.device)
        a = self._args
        a.lr_dev, a.grad_scale = None, None
        if isinstance(lr, torch.Tensor):
            a.lr_dev, a.lr = self._scalar("lr", lr), 0.0
        else:
            a.lr = self.lr if lr is None else float(lr)
        if grad_scale is not None:
            a.grad_scale = self._scalar("grad_scale", grad_scale)
        handle = _raw_stream(stream, self._index)
        rlk_muon_step(self._list, a, _workspace(self, self._ws_bytes, stream, handle), handle)

    def _scalar(self, name, t):
        import torch
        if t.dtype != torch.float32 or t.numel() != 1 or t.device != self.device:
            raise ValueError(f"{name} must be one float32 value on {self.device}")
        return t.data_ptr()
