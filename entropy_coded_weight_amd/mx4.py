"""Microscaled 4-bit matrices and the 4-bit key/value cache of libecw.so.

The format and the operations are described in include/ecw.h; operands are checked and
results allocated in the native binding (csrc/mx4_bind.cpp).  Inference only: no call
records a gradient, and an input that requires one is used as its values.

    w = mx4_quantize(weights)                  # MX4Tensor, 4.25 bits per element
    y = w.gemm(x)                              # x: fp16/bf16 [batch, cols] -> fp32 [batch, rows]
    y = w.gemm(mx4_quantize(x))                # both operands in 4 bits

    cache = KV4Cache(pages, kv_heads, head_dim)
    cache.append(k, v, page_table, lens)       # the last rows of each sequence
    o = cache.attend(q, page_table, lens)      # causal attention over the cache

Work runs on the current stream of the operands' device, or on `stream`, one of the same
device; results are allocated there.  Whoever passes a stream orders it after the producers of the operands.
"""
from __future__ import annotations

import ctypes
import os

import torch

from . import EcwError, _check, lib

_BIND_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_mx4.so")


class _Cache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p)] + [(n, ctypes.c_uint32) for n in (
        "pages", "kv_heads", "head_dim", "page_tokens")]


_bound = None


def _native():
    """The binding, with the library loaded (raises if they have not been built)."""
    global _bound
    if _bound is None:
        L = lib()
        if not os.path.exists(_BIND_PATH):
            raise ImportError(f"{_BIND_PATH} missing: run __graft_entry__.build() (or "
                              "python entropy_coded_weight_amd/build.py) first")
        from . import _mx4
        L.kv4_bytes.argtypes = [ctypes.POINTER(_Cache), ctypes.POINTER(ctypes.c_size_t)]
        L.kv4_bytes.restype = ctypes.c_int
        _mx4.init(L._name, EcwError)
        _bound = _mx4
    return _bound


def _on(stream, tensors, call):
    """call() with `stream` current; the tensors live on until its work is done."""
    tensors = [t for t in tensors if isinstance(t, torch.Tensor) and t.is_cuda]
    for t in tensors:  # work goes to the tensors' device, whose current stream would be another one
        if t.device != stream.device:
            raise ValueError(f"the stream is on {stream.device}, an operand on {t.device}")
    with torch.cuda.stream(stream):
        for t in tensors:
            t.record_stream(stream)
        return call()


class MX4Tensor:
    """A matrix [rows, cols] of 4-bit floats with a power-of-two scale per 32 columns.

    codes: uint8 [rows, 64 * ceil(cols / 128)], scales: uint8 [rows, 16 * ceil(cols / 512)]
    (the byte of each block's scale; 255: the block is NaN)."""

    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes, scales, rows, cols):
        for name, t, width in (("codes", codes, (cols + 127) // 128 * 64), ("scales", scales, (cols + 511) // 512 * 16)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda:
                raise TypeError(f"{name} must be a cuda tensor")
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
        if stream is not None:
            return _on(stream, (self.codes, self.scales, out), lambda: self.dequantize(dtype, out))
        return _native().dequantize(self.codes, self.scales, self.cols, dtype, out)

    def gemm(self, x, y=None, out_dtype=torch.float32, stream=None) -> torch.Tensor:
        """y = x W^T for any batch: x fp16/bf16 [batch, cols] (or [cols]) or an MX4Tensor
        [batch, cols]; y [batch, rows], fp32 unless out_dtype (fp16, bf16) says otherwise."""
        if stream is not None:
            used = (x.codes, x.scales) if isinstance(x, MX4Tensor) else (x,)
            return _on(stream, (self.codes, self.scales, y, *used), lambda: self.gemm(x, y, out_dtype))
        if isinstance(x, MX4Tensor):
            return _native().gemm_mx4(self.codes, self.scales, self.cols, x.codes, x.scales, x.cols, y, out_dtype)
        return _native().gemm(self.codes, self.scales, self.cols, x, y, out_dtype)


def mx4_quantize(x: torch.Tensor, out: MX4Tensor | None = None, stream=None) -> MX4Tensor:
    """x fp16/bf16/fp32 [rows, cols] (or [cols]), rows at any stride, as an MX4Tensor."""
    if stream is not None:
        used = (x,) if out is None else (x, out.codes, out.scales)
        return _on(stream, used, lambda: mx4_quantize(x, out))
    if out is not None:
        if not isinstance(x, torch.Tensor) or out.shape != (tuple(x.shape) if x.dim() == 2 else (1, *x.shape)):
            raise ValueError(f"out is {out.shape}, x {getattr(x, 'shape', x)}")
        _native().quantize(x, out.codes, out.scales)
        return out
    t = MX4Tensor.__new__(MX4Tensor)
    t.codes, t.scales, t.cols = _native().quantize(x, None, None)
    t.rows = t.codes.shape[0]
    return t


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
        _native()
        n = ctypes.c_size_t(0)
        _check(lib().kv4_bytes(_Cache(None, pages, kv_heads, head_dim, page_tokens), n), "kv4_bytes")
        self.data = torch.zeros(n.value, dtype=torch.uint8, device=device)
        if not self.data.is_cuda:
            raise TypeError("the cache must be on a cuda device")
        self.pages, self.kv_heads, self.head_dim, self.page_tokens = pages, kv_heads, head_dim, page_tokens
        self._as_args = (self.data, pages, kv_heads, head_dim, page_tokens)

    @property
    def device(self):
        return self.data.device

    def append(self, k, v, page_table, lens, starts=None, stream=None) -> None:
        """k, v fp16/bf16/fp32 [rows, kv_heads, head_dim] into the cache; rows without a
        page are dropped.  Calls on different streams that write the same pages race."""
        if stream is not None:
            return _on(stream, (self.data, k, v, page_table, lens, starts),
                       lambda: self.append(k, v, page_table, lens, starts))
        return _native().append(*self._as_args, k, v, page_table, lens, starts)

    def read(self, page_table, lens, rows: int, starts=None, dtype=torch.bfloat16, stream=None):
        """The values of the last rows of each sequence as (k, v) [rows, kv_heads, head_dim];
        zeros for a row without a page."""
        if stream is not None:
            return _on(stream, (self.data, page_table, lens, starts),
                       lambda: self.read(page_table, lens, rows, starts, dtype))
        return _native().read(*self._as_args, page_table, lens, starts, rows, dtype)

    def attend(self, q, page_table, lens, starts=None, max_rows=None, max_len=None, window: int = 0, sinks: int = 0,
               scale=None, out=None, stream=None) -> torch.Tensor:
        """softmax(scale q k^T) v, causal, over the cache's tokens of each row's sequence.

        q fp16/bf16 [rows, q_heads, head_dim]; q_heads a multiple of kv_heads.  A row at
        position p sees tokens up to p; with a window only the last `window` of them and
        the sequence's first `sinks`.  A row that sees nothing gives zeros.  Softmax weights
        are rounded to q's type, sums are fp32; with q in fp16, keys and values past fp16's
        range count as NaN.  scale: head_dim ** -0.5.  max_rows, max_len: the most rows and tokens of one sequence, if
        the host knows them; they shape the launch, not the result's meaning."""
        if stream is not None:
            return _on(stream, (self.data, q, page_table, lens, starts, out),
                       lambda: self.attend(q, page_table, lens, starts, max_rows, max_len, window, sinks, scale, out))
        return _native().attend(*self._as_args, q, page_table, lens, starts, max_rows, max_len, window, sinks, scale,
                                out)
