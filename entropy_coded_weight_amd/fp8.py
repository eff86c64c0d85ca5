"""Block-scaled 8-bit matrices, the root-mean-square norm and the rotary positions of libecw.so.

The format and the operations are described in include/ecw.h; operands are checked and
results allocated in the native binding (csrc/fp8_bind.cpp).  Inference only: no call
records a gradient, and an input that requires one is used as its values.

    w = fp8_quantize(weights)                      # FP8Tensor, 8.0625 bits per element
    h, x = rms_norm(y, weight, residual=x, out_dtype=torch.float8_e4m3fn)
    y = w.gemm(h, out_dtype=torch.bfloat16)        # both operands in 8 bits
    a = fp8_quantize(up, gate=gate)                # silu(gate) * up, for the down projection

    rotary = Rotary(head_dim, base=500000.0)
    q, k = rotary(q, k, positions)

Work runs on the current stream of the operands' device, or on `stream`, one of the same
device; results are allocated there.  Whoever passes a stream orders it after the producers of the operands.
A given output that overlaps an operand is refused, but where a call says that it works in place.
"""
from __future__ import annotations

import torch

from ._binding import native, on


class FP8Tensor:
    """A matrix [rows, cols] of E4M3 numbers with a power-of-two scale per 128 columns of a row.

    codes: uint8 [rows, 128 * ceil(cols / 128)], scales: uint8 [rows, 16 * ceil(cols / 2048)]
    (the byte of each block's scale; 255: the block is NaN)."""

    __slots__ = ("codes", "scales", "rows", "cols")

    def __init__(self, codes, scales, rows, cols):
        for name, t, width in (("codes", codes, (cols + 127) // 128 * 128), ("scales", scales, (cols + 2047) // 2048 * 16)):
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
            return on(stream, (self.codes, self.scales, out), lambda: self.dequantize(dtype, out))
        return native("_fp8").dequantize(self.codes, self.scales, self.cols, dtype, out)

    def gemm(self, x: FP8Tensor, y=None, out_dtype=torch.float32, stream=None, short_sums: bool = False) -> torch.Tensor:
        """y = x W^T for any batch: x an FP8Tensor [batch, cols]; y [batch, rows], fp32 unless
        out_dtype (fp16, bf16) says otherwise; one that is given starts at a multiple of 16 bytes.

        Products are exact, sums fp32, in an order that depends on the shape, and rounded once.
        short_sums, for 16-bit results: up to 16 neighbouring products may be added with 12
        fraction bits under the largest one's power of two first, in about half the time for
        many rows.  A sum is then off by up to 2^-8 of its products' magnitudes (1.5e-5 to 7e-5
        of the result in 2-norm measured on normal numbers and with large columns): not where
        large products cancel."""
        if not isinstance(x, FP8Tensor):
            raise TypeError("x must be an FP8Tensor: fp8_quantize(x), or a norm's 8-bit output")
        if stream is not None:
            return on(stream, (self.codes, self.scales, y, x.codes, x.scales),
                      lambda: self.gemm(x, y, out_dtype, short_sums=short_sums))
        return native("_fp8").gemm(self.codes, self.scales, self.cols, x.codes, x.scales, x.cols, y, out_dtype, short_sums)


def _tensor(codes, scales, cols):
    t = FP8Tensor.__new__(FP8Tensor)
    t.codes, t.scales, t.rows, t.cols = codes, scales, codes.shape[0], cols
    return t


def _fits(out, x):
    if not isinstance(out, FP8Tensor):
        raise TypeError("out must be an FP8Tensor")
    if not isinstance(x, torch.Tensor) or out.shape != (tuple(x.shape) if x.dim() == 2 else (1, *x.shape)):
        raise ValueError(f"out is {out.shape}, x {getattr(x, 'shape', x)}")


def fp8_quantize(x: torch.Tensor, gate: torch.Tensor | None = None, out: FP8Tensor | None = None,
                 stream=None) -> FP8Tensor:
    """x fp16/bf16/fp32 [rows, cols] (or [cols]), rows at any stride, as an FP8Tensor; with a
    gate of x's shape and dtype, silu(gate) * x."""
    if out is not None:
        _fits(out, x)
    if stream is not None:
        used = (x, gate) if out is None else (x, gate, out.codes, out.scales)
        return on(stream, used, lambda: fp8_quantize(x, gate, out))
    if out is not None:
        native("_fp8").quantize(x, gate, out.codes, out.scales)
        return out
    return _tensor(*native("_fp8").quantize(x, gate, None, None))


def rms_norm(x: torch.Tensor, weight: torch.Tensor | None = None, residual: torch.Tensor | None = None,
             eps: float = 1e-6, out=None, out_dtype=None, residual_out: torch.Tensor | None = None, stream=None):
    """h / sqrt(mean(h^2) + eps) * weight over the rows of h = x + residual.

    x fp16/bf16/fp32 [rows, cols] (or [cols]), rows at any stride, up to 32768 columns; weight
    [cols]; residual of x's shape, in x's dtype or fp32.  The result has x's dtype, or
    out_dtype: fp16, bf16, fp32, or torch.float8_e4m3fn for an FP8Tensor.  With a residual
    the call gives (result, h), h in the residual's dtype; residual_out=residual writes it
    in place.  h is rounded once, into that; the result is made of the unrounded h."""
    if stream is not None:
        used = (out.codes, out.scales) if isinstance(out, FP8Tensor) else (out,)
        return on(stream, (x, weight, residual, residual_out, *used),
                  lambda: rms_norm(x, weight, residual, eps, out, out_dtype, residual_out))
    if isinstance(out, FP8Tensor):
        _fits(out, x)
        *_, h = native("_fp8").rms_norm(x, weight, residual, eps, None, out.codes, out.scales, residual_out)
        return out if residual is None else (out, h)
    if out_dtype is torch.float8_e4m3fn:
        if out is not None:
            raise TypeError("out must be an FP8Tensor for an 8-bit result")
        *t, h = native("_fp8").rms_norm(x, weight, residual, eps, None, None, None, residual_out)
        return _tensor(*t) if residual is None else (_tensor(*t), h)
    if out_dtype is None:
        out_dtype = x.dtype if isinstance(x, torch.Tensor) else torch.float32  # no tensor: refused by the binding
    return native("_fp8").rms_norm(x, weight, residual, eps, out_dtype, out, None, residual_out)


class Rotary:
    """Rotary positions on one axis or several (time, height, width).

    Pair j of a head's first rotary_dim dimensions is turned by position * inv_freq[j]:
    dimensions j and j + rotary_dim / 2, or with `neighbours` 2 j and 2 j + 1.  inv_freq
    (rotary_dim / 2 numbers, used as their float64 values): base ** (-2 j / rotary_dim).
    With several axes each pair follows the position on one: `sections` says how many pairs
    each axis has, one after the other, `axes` the axis of every pair.  scale multiplies
    what is turned.  Angles are within 2^-32 of a turn for positions up to 2^32 of either sign,
    and within 2^-64 of it times the position beyond, so negated positions undo a turn (and give
    the gradient of one)."""

    def __init__(self, head_dim: int, rotary_dim: int | None = None, base: float = 10000.0, inv_freq=None,
                 sections=None, axes=None, neighbours: bool = False, scale: float = 1.0, device="cuda"):
        rotary_dim = head_dim if rotary_dim is None else rotary_dim
        if not 0 < head_dim <= 4096 or not 0 < rotary_dim <= head_dim or rotary_dim % 2:
            raise ValueError(f"rotary_dim must be even, in [2, head_dim], head_dim at most 4096: got {rotary_dim} of {head_dim}")
        pairs = rotary_dim // 2
        if inv_freq is None:
            if not base > 0:
                raise ValueError("base must be positive")
            inv_freq = [base ** (-2 * j / rotary_dim) for j in range(pairs)]
        inv_freq = [float(f) for f in inv_freq]
        if sections is not None and axes is not None:
            raise ValueError("sections and axes say the same: pass one")
        if sections is not None:
            if any(n < 0 for n in sections):
                raise ValueError("sections must not be negative")
            axes = [i for i, n in enumerate(sections) for _ in range(n)]
            count = len(sections)
        else:
            axes = [0] * pairs if axes is None else [int(i) for i in axes]
            count = max(axes, default=0) + 1
        if len(inv_freq) != pairs or len(axes) != pairs:
            raise ValueError(f"{len(inv_freq)} frequencies and axes for {len(axes)} pairs, expected {pairs}")
        if not 0 < count <= 255 or min(axes) < 0:
            raise ValueError("axes must be in [0, 255)")
        self.head_dim, self.rotary_dim, self.axes, self.neighbours, self.scale = head_dim, rotary_dim, count, neighbours, scale
        # as fractions of a turn in 2^-64, modulo a turn
        turns = [_turn(f) for f in inv_freq]
        self.freqs = torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)
        self.axis_of = torch.tensor(axes, dtype=torch.uint8, device=device)
        if not self.freqs.is_cuda:
            raise TypeError("the frequencies must be on a cuda device")

    def __call__(self, q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, out=None, stream=None):
        """q [rows, heads, head_dim] and k (or None), fp16/bf16/fp32 at any strides of rows and
        heads, turned by positions, int32 or int64 [rows] or [axes, rows].  Gives (q, k), or q
        alone; out=(q, k) writes in place."""
        q_out, k_out = (None, None) if out is None else (out, None) if isinstance(out, torch.Tensor) else out
        if stream is not None:
            return on(stream, (q, k, positions, self.freqs, self.axis_of, q_out, k_out), lambda: self(q, k, positions, (q_out, k_out)))
        return native("_fp8").rotary(q, k, positions, self.freqs, self.axis_of, self.axes, self.head_dim, self.neighbours,
                                     self.scale, q_out, k_out)


# 2 pi to 40 digits, as a fraction
_TWO_PI = (62831853071795864769252867665590057683943, 10 ** 40)


def _turn(f: float) -> int:
    """f radians as a fraction of a turn in 2^-64, modulo a turn, rounded to nearest."""
    if f != f or f in (float("inf"), float("-inf")):
        raise ValueError("frequencies must be finite")
    num, den = f.as_integer_ratio()
    num, den = num * _TWO_PI[1] << 64, den * _TWO_PI[0]
    return (2 * num + den) // (2 * den) % (1 << 64)
