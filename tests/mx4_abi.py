"""The 4-bit entry points of libecw.so through ctypes, as include/ecw.h declares them."""
import ctypes

import entropy_coded_weight_amd as ecw


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_uint32) for n in (
        "pages", "kv_heads", "head_dim", "page_tokens")]


class _Rows(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("starts", ctypes.c_void_p)] + [(n, ctypes.c_uint32) for n in ("batch", "table_width", "rows")]


class _Attention(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("q_heads", "max_rows", "max_len", "window", "sinks")] + [
        ("scale", ctypes.c_float)]


def _lib():
    L = ctypes.CDLL(ecw.lib()._name)  # a handle of its own: the binding's signatures stay as they are
    vp, u32, i32, i64, sz = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    P = ctypes.POINTER
    L.mx4_quantize.argtypes = [vp, vp, i32, i64, u32, u32, vp, vp]
    L.mx4_dequantize.argtypes = [vp, vp, vp, u32, u32, vp, i32]
    L.mx4_gemm.argtypes = [vp, vp, vp, u32, u32, vp, i32, i64, u32, vp, i32]
    L.mx4_gemm_mx4.argtypes = [vp, vp, vp, u32, u32, vp, vp, u32, vp, i32]
    L.kv4_bytes.argtypes = [P(_Cache), P(sz)]
    L.kv4_append.argtypes = [vp, P(_Cache), P(_Rows), vp, vp, i32, P(i64)]
    L.kv4_read.argtypes = [vp, P(_Cache), P(_Rows), vp, vp, i32]
    L.kv4_attend_workspace_size.argtypes = [P(_Cache), P(_Rows), P(_Attention), P(sz)]
    L.kv4_attend.argtypes = [vp, P(_Cache), P(_Rows), P(_Attention), vp, i32, i64, i64, vp, vp, sz]
    L.ecw_last_error.restype = ctypes.c_char_p
    return L
