"""The 8-bit, norm and rotary entry points of libecw.so through ctypes, as include/ecw.h declares them."""
import ctypes

import entropy_coded_weight_amd as ecw

_vp, _u32, _i32, _i64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int, ctypes.c_int64


class Norm(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("x", "residual", "weight", "residual_out", "y", "y_scales")]
                + [(n, _i64) for n in ("x_stride", "residual_stride", "residual_out_stride")]
                + [(n, _u32) for n in ("rows", "cols")]
                + [(n, _i32) for n in ("x_dtype", "residual_dtype", "weight_dtype", "y_dtype")] + [("eps", ctypes.c_float)])


class Rotary(ctypes.Structure):
    _fields_ = ([(n, _vp) for n in ("q", "k", "q_out", "k_out", "positions", "freqs", "axis_of")]
                + [(n, _i64) for n in ("q_row", "q_head", "k_row", "k_head", "q_out_row", "q_out_head", "k_out_row",
                                       "k_out_head", "axis_stride")]
                + [(n, _u32) for n in ("rows", "q_heads", "k_heads", "head_dim", "rotary_dim", "axes")]
                + [(n, _i32) for n in ("dtype", "neighbours", "wide_positions")] + [("scale", ctypes.c_float)])


def _lib():
    L = ctypes.CDLL(ecw.lib()._name)  # a handle of its own: the binding's signatures stay as they are
    L.fp8_quantize.argtypes = [_vp, _vp, _i32, _i64, _vp, _i64, _u32, _u32, _vp, _vp]
    L.fp8_dequantize.argtypes = [_vp, _vp, _vp, _u32, _u32, _vp, _i32]
    L.fp8_gemm_workspace_size.argtypes = [_u32, _u32, _u32, _i32, ctypes.POINTER(ctypes.c_size_t)]
    L.fp8_gemm.argtypes = [_vp, _vp, _vp, _u32, _u32, _vp, _vp, _u32, _vp, _i32, _vp, ctypes.c_size_t]
    L.rms_norm.argtypes = [_vp, ctypes.POINTER(Norm)]
    L.rotary_apply.argtypes = [_vp, ctypes.POINTER(Rotary)]
    L.ecw_last_error.restype = ctypes.c_char_p
    return L
