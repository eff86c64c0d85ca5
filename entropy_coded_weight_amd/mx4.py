"""Microscaled 4-bit matrices and the 4-bit key/value cache of libecw.so.

Argument checks and marshalling only; the format and the operations are described in
include/ecw.h.  Inference only: no call records a gradient.

    w = mx4_quantize(weights)                  # MX4Tensor, 4.25 bits per element
    y = w.gemm(x)                              # x: fp16/bf16 [batch, cols] -> fp32 [batch, rows]
    y = w.gemm(mx4_quantize(x))                # both operands in 4 bits

    cache = KV4Cache(pages, kv_heads, head_dim)
    cache.append(k, v, page_table, lens)       # the last rows of each sequence
    o = cache.attend(q, page_table, lens)      # causal attention over the cache

Work runs on the current stream of the operands' device, or on `stream`; results are
allocated there.  Whoever passes a stream orders it after the producers of the operands.
"""
from __future__ import annotations

import ctypes

import torch

from . import DT_BF16, DT_F16, DT_F32, _check, lib

_FLOATS = {torch.float16: DT_F16, torch.bfloat16: DT_BF16, torch.float32: DT_F32}
_raw_stream = torch._C._cuda_getCurrentRawStream


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_uint32) for n in (
        "pages", "kv_heads", "head_dim", "page_tokens")]


class _Rows(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("starts", ctypes.c_void_p)] + [(n, ctypes.c_uint32) for n in ("batch", "table_width", "rows")]


class _Attention(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint32) for n in ("q_heads", "max_rows", "max_len", "window", "sinks")] + [
        ("scale", ctypes.c_float)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
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
        for f in ("mx4_quantize", "mx4_dequantize", "mx4_gemm", "mx4_gemm_mx4", "kv4_bytes", "kv4_append", "kv4_read",
                  "kv4_attend_workspace_size", "kv4_attend"):
            getattr(L, f).restype = ctypes.c_int
        _bound = L
    return _bound


_get_device = torch._C._cuda_getDevice


def _elsewhere(device, stream, tensors, call):
    """call() with `device` and `stream` current; the tensors live on until its work is done."""
    with torch.cuda.device(device), torch.cuda.stream(stream):
        if stream is not None:
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        return call()


def _on_gpu(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a cuda tensor")


def _float(t, name, dtypes=_FLOATS):
    d = dtypes.get(t.dtype)
    if d is None:
        raise TypeError(f"{name} must be " + ", ".join(str(d).replace("torch.", "") for d in dtypes))
    return d


_HALVES = {torch.float16: DT_F16, torch.bfloat16: DT_BF16}


def _bad_ints(t, name, device, shape):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != device:
        raise TypeError(f"{name} must be an int32 tensor on {device}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    raise TypeError(f"{name} must have a unit inner stride")


_I32 = torch.int32


class MX4Tensor:
    """A matrix [rows, cols] of 4-bit floats with a power-of-two scale per 32 columns.

    codes: uint8 [rows, 64 * ceil(cols / 128)], scales: uint8 [rows, 16 * ceil(cols / 512)]
    (the byte of each block's scale; 255: the block is NaN)."""

    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes, scales, rows, cols):
        for name, t, width in (("codes", codes, (cols + 127) // 128 * 64), ("scales", scales, (cols + 511) // 512 * 16)):
            _on_gpu(t, name)
            if t.dtype != torch.uint8 or not t.is_contiguous():
                raise TypeError(f"{name} must be contiguous uint8")
            if tuple(t.shape) != (rows, width):
                raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(rows, width)}")
        if scales.device != codes.device:
            raise ValueError("codes and scales are on different devices")
        self.codes, self.scales, self.rows, self.cols = codes, scales, rows, cols

    @property
    def shape(self):
        return self.rows, self.cols

    @property
    def device(self):
        return self.codes.device

    def stored_bytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def dequantize(self, dtype=torch.float16, out=None, stream=None) -> torch.Tensor:
        """The values as a dense [rows, cols] matrix: exact in bfloat16 and float32."""
        dev = self.codes.device
        if stream is not None or dev.index != _get_device():
            return _elsewhere(dev, stream, (self.codes, self.scales, out), lambda: self.dequantize(dtype, out))
        if out is None:
            out = torch.empty((self.rows, self.cols), dtype=dtype, device=dev)
        elif tuple(out.shape) != (self.rows, self.cols) or not out.is_contiguous() or out.device != dev:
            raise ValueError(f"out must be a contiguous {(self.rows, self.cols)} tensor on {dev}")
        _check(_lib().mx4_dequantize(_raw_stream(dev.index), self.codes.data_ptr(), self.scales.data_ptr(), self.rows,
                                     self.cols, out.data_ptr(), _float(out, "out")), "mx4_dequantize")
        return out

    def gemm(self, x, y=None, out_dtype=torch.float32, stream=None) -> torch.Tensor:
        """y = x W^T for any batch: x fp16/bf16 [batch, cols] (or [cols]) or an MX4Tensor
        [batch, cols]; y [batch, rows], fp32 unless out_dtype (fp16, bf16) says otherwise."""
        dev = self.codes.device
        both = isinstance(x, MX4Tensor)
        if both:
            batch, cols = x.rows, x.cols
        else:
            _on_gpu(x, "x")
            if x.dim() == 1:
                x = x.unsqueeze(0)
            if x.dim() != 2:
                raise ValueError("x must be [batch, cols]")
            batch, cols = x.shape
        if cols != self.cols:
            raise ValueError(f"x has {cols} columns, the tensor {self.cols}")
        if x.device != dev:
            raise ValueError(f"x is on {x.device}, the tensor on {dev}")
        if stream is not None or dev.index != _get_device():
            used = (x.codes, x.scales) if both else (x,)
            return _elsewhere(dev, stream, (self.codes, self.scales, y, *used), lambda: self.gemm(x, y, out_dtype))
        if y is None:
            y = torch.empty((batch, self.rows), dtype=out_dtype, device=dev)
        elif tuple(y.shape) != (batch, self.rows) or not y.is_contiguous() or y.device != dev:
            raise ValueError(f"y must be a contiguous {(batch, self.rows)} tensor on {dev}")
        yd = _float(y, "y")
        if both:
            _check(_lib().mx4_gemm_mx4(_raw_stream(dev.index), self.codes.data_ptr(), self.scales.data_ptr(),
                                       self.rows, cols, x.codes.data_ptr(), x.scales.data_ptr(), batch, y.data_ptr(),
                                       yd), "mx4_gemm_mx4")
            return y
        xd = _float(x, "x", _HALVES)
        if cols > 1 and x.stride(1) != 1:
            raise TypeError("x must have a unit inner stride")
        _check(_lib().mx4_gemm(_raw_stream(dev.index), self.codes.data_ptr(), self.scales.data_ptr(), self.rows, cols,
                               x.data_ptr(), xd, x.stride(0), batch, y.data_ptr(), yd), "mx4_gemm")
        return y


def mx4_quantize(x: torch.Tensor, out: MX4Tensor | None = None, stream=None) -> MX4Tensor:
    """x fp16/bf16/fp32 [rows, cols] (or [cols]), rows at any stride, as an MX4Tensor."""
    _on_gpu(x, "x")
    if x.dim() == 1:
        x = x.unsqueeze(0)
    if x.dim() != 2 or x.shape[1] == 0:
        raise ValueError("x must be [rows, cols] with at least one column")
    xd = _float(x, "x")
    rows, cols = x.shape
    if cols > 1 and x.stride(1) != 1:
        raise TypeError("x must have a unit inner stride")
    dev = x.device
    if stream is not None or dev.index != _get_device():
        used = (x,) if out is None else (x, out.codes, out.scales)
        return _elsewhere(dev, stream, used, lambda: mx4_quantize(x, out))
    if out is None:
        out = MX4Tensor.__new__(MX4Tensor)
        out.codes = torch.empty((rows, (cols + 127) // 128 * 64), dtype=torch.uint8, device=dev)
        out.scales = torch.empty((rows, (cols + 511) // 512 * 16), dtype=torch.uint8, device=dev)
        out.rows, out.cols = rows, cols
    elif out.shape != (rows, cols) or out.device != dev:
        raise ValueError(f"out must be a {(rows, cols)} MX4Tensor on {dev}")
    _check(_lib().mx4_quantize(_raw_stream(dev.index), x.data_ptr(), xd, x.stride(0), rows, cols,
                               out.codes.data_ptr(), out.scales.data_ptr()), "mx4_quantize")
    return out


class KV4Cache:
    """Keys and values of many sequences in 4 bits, in pages of page_tokens tokens.

    Which pages a sequence owns is the caller's: page_table int32 [batch, width] (an entry
    outside 0..pages-1 is no page), lens int32 [batch] the tokens of each sequence with
    the call's rows among them.  The rows of a call are each sequence's last ones, in
    order: rows / batch of each, or starts int32 [batch + 1] their first rows.  All three
    stay on the device; bad values there reach no memory outside the cache."""

    def __init__(self, pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda"):
        for name, v in (("pages", pages), ("kv_heads", kv_heads), ("head_dim", head_dim), ("page_tokens", page_tokens)):
            if not 0 < v < 1 << 31:
                raise ValueError(f"{name} must be positive")
        self._c = _Cache(None, pages, kv_heads, head_dim, page_tokens)
        n = ctypes.c_size_t(0)
        _check(_lib().kv4_bytes(ctypes.byref(self._c), ctypes.byref(n)), "kv4_bytes")
        self.data = torch.zeros(n.value, dtype=torch.uint8, device=device)
        _on_gpu(self.data, "cache")
        self._c.data = self.data.data_ptr()
        self.pages, self.kv_heads, self.head_dim, self.page_tokens = pages, kv_heads, head_dim, page_tokens
        self.device = self.data.device
        self._plans = {}

    def _rows(self, page_table, lens, starts, rows):
        dev = self.device
        if (not isinstance(page_table, torch.Tensor) or page_table.dtype is not _I32 or page_table.device != dev
                or page_table.dim() != 2):
            _bad_ints(page_table, "page_table", dev, ("batch", "width"))
        batch, width = page_table.shape
        stride, inner = page_table.stride()
        if inner != 1 and width > 1 and batch:
            _bad_ints(page_table, "page_table", dev, (batch, width))
        if (not isinstance(lens, torch.Tensor) or lens.dtype is not _I32 or lens.device != dev
                or lens.shape != (batch,) or not lens.is_contiguous()):
            _bad_ints(lens, "lens", dev, (batch,))
        first = None
        if starts is not None:
            if (not isinstance(starts, torch.Tensor) or starts.dtype is not _I32 or starts.device != dev
                    or starts.shape != (batch + 1,) or not starts.is_contiguous()):
                _bad_ints(starts, "starts", dev, (batch + 1,))
            first = starts.data_ptr()
        elif rows and (batch == 0 or rows % batch):
            raise ValueError(f"{rows} rows are not the same number for each of {batch} sequences: pass starts")
        return _Rows(page_table.data_ptr(), stride, lens.data_ptr(), first, batch, width, rows)

    def _heads(self, t, name, heads=None):
        if not isinstance(t, torch.Tensor) or t.device != self.device:
            _on_gpu(t, name)
            raise ValueError(f"{name} is on {t.device}, the cache on {self.device}")
        if t.dim() != 3 or t.shape[2] != self.head_dim or (heads and t.shape[1] != heads):
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected (*, {heads or '*'}, {self.head_dim})")
        if t.stride(2) != 1:
            raise TypeError(f"{name} must have a unit inner stride")

    def append(self, k, v, page_table, lens, starts=None, stream=None) -> None:
        """k, v fp16/bf16/fp32 [rows, kv_heads, head_dim] into the cache; rows without a
        page are dropped.  Calls on different streams that write the same pages race."""
        self._heads(k, "k", self.kv_heads)
        self._heads(v, "v", self.kv_heads)
        if k.shape[0] != v.shape[0] or k.dtype != v.dtype:
            raise ValueError("k and v must agree in rows and dtype")
        dt = _float(k, "k")
        dev = self.device
        r = self._rows(page_table, lens, starts, k.shape[0])
        if stream is not None or dev.index != _get_device():
            return _elsewhere(dev, stream, (self.data, k, v, page_table, lens, starts),
                              lambda: self.append(k, v, page_table, lens, starts))
        strides = (ctypes.c_int64 * 4)(k.stride(0), k.stride(1), v.stride(0), v.stride(1))
        _check(_lib().kv4_append(_raw_stream(dev.index), self._c, r, k.data_ptr(), v.data_ptr(), dt, strides),
               "kv4_append")

    def read(self, page_table, lens, rows: int, starts=None, dtype=torch.bfloat16, stream=None):
        """The values of the last rows of each sequence as (k, v) [rows, kv_heads, head_dim];
        zeros for a row without a page."""
        if rows < 0:
            raise ValueError("rows must not be negative")
        dev = self.device
        r = self._rows(page_table, lens, starts, rows)
        if stream is not None or dev.index != _get_device():
            return _elsewhere(dev, stream, (self.data, page_table, lens, starts),
                              lambda: self.read(page_table, lens, rows, starts, dtype))
        k = torch.empty((rows, self.kv_heads, self.head_dim), dtype=dtype, device=dev)
        v = torch.empty_like(k)
        _check(_lib().kv4_read(_raw_stream(dev.index), self._c, r, k.data_ptr(), v.data_ptr(), _float(k, "dtype")),
               "kv4_read")
        return k, v

    def attend(self, q, page_table, lens, starts=None, max_rows=None, max_len=None, window: int = 0, sinks: int = 0,
               scale=None, out=None, stream=None) -> torch.Tensor:
        """softmax(scale q k^T) v, causal, over the cache's tokens of each row's sequence.

        q fp16/bf16 [rows, q_heads, head_dim]; q_heads a multiple of kv_heads.  A row at
        position p sees tokens up to p; with a window only the last `window` of them and
        the sequence's first `sinks`.  A row that sees nothing gives zeros.  scale:
        head_dim ** -0.5.  max_rows, max_len: the most rows and tokens of one sequence, if
        the host knows them; they shape the launch, not the result's meaning."""
        self._heads(q, "q")
        dt = _float(q, "q", _HALVES)
        rows, q_heads, dim = q.shape
        if q_heads == 0 or q_heads % self.kv_heads:
            raise ValueError(f"{q_heads} query heads are no multiple of {self.kv_heads} key/value heads")
        if window < 0 or sinks < 0 or (max_rows or 0) < 0 or (max_len or 0) < 0:
            raise ValueError("window, sinks, max_rows and max_len must not be negative")
        dev = self.device
        r = self._rows(page_table, lens, starts, rows)
        if stream is not None or dev.index != _get_device():
            return _elsewhere(dev, stream, (self.data, q, page_table, lens, starts, out),
                              lambda: self.attend(q, page_table, lens, starts, max_rows, max_len, window, sinks,
                                                  scale, out))
        if out is None:
            out = torch.empty((rows, q_heads, dim), dtype=q.dtype, device=dev)
        elif tuple(out.shape) != tuple(q.shape) or not out.is_contiguous() or out.dtype != q.dtype or out.device != dev:
            raise ValueError(f"out must be a contiguous {tuple(q.shape)} {q.dtype} tensor on {dev}")
        L = _lib()
        # the attention's description and workspace by its sizes, which a decode loop repeats
        key = (rows, q_heads, r.batch, r.table_width, max_rows, max_len, window, sinks, scale)
        plan = self._plans.get(key)
        if plan is None:
            top = 1 << 30
            a = _Attention(q_heads, min(max_rows or 0, top), min(max_len or 0, top), min(window, top),
                           min(sinks, top), dim ** -0.5 if scale is None else scale)
            n = ctypes.c_size_t(0)
            _check(L.kv4_attend_workspace_size(self._c, r, a, n), "kv4_attend_workspace_size")
            if len(self._plans) >= 64:
                self._plans.clear()
            plan = self._plans[key] = a, n.value
        a, n = plan
        ws = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
        _check(L.kv4_attend(_raw_stream(dev.index), self._c, r, a, q.data_ptr(), dt, q.stride(0), q.stride(1),
                            out.data_ptr(), ws.data_ptr() if n else None, n), "kv4_attend")
        return out
