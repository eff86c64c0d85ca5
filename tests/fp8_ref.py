"""The block-scaled 8-bit format, the norm and the rotary positions in float64 numpy, from
their definitions."""
import numpy as np


def _levels():
    """The 127 magnitudes of E4M3, by code."""
    out = []
    for c in range(127):
        e, m = c >> 3, c & 7
        out.append(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
    return np.array(out)


LEVELS = _levels()
MIDDLES = (LEVELS[1:] + LEVELS[:-1]) / 2


def quantise(x):
    """x [..., cols] -> codes uint8 [..., cols up to 128], scale bytes [..., blocks]."""
    x = np.asarray(x, np.float64)
    pad = -x.shape[-1] % 128
    x = np.concatenate([x, np.zeros((*x.shape[:-1], pad))], -1)
    x = x.reshape(*x.shape[:-1], x.shape[-1] // 128, 128)
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(top)
    s = np.zeros(top.shape, np.int64)
    ok = ~bad & (top > 0)
    s[ok] = np.ceil(np.log2(top[ok] / 448)).astype(np.int64)
    s[ok] += top[ok] > 448 * np.exp2(s[ok].astype(np.float64))           # where the logarithm was rounded
    s[ok] -= top[ok] <= 448 * np.exp2(s[ok].astype(np.float64) - 1)
    s = np.clip(s, -117, 119)
    a = np.abs(np.where(bad[..., None], 0, x)) * np.exp2(-s.astype(np.float64))[..., None]
    lo = np.searchsorted(MIDDLES, a, side="left")    # a tie goes down
    hi = np.searchsorted(MIDDLES, a, side="right")   # a tie goes up
    code = np.where(lo % 2 == 0, lo, hi)
    code = np.where(lo == hi, lo, code) + 128 * np.signbit(np.where(bad[..., None], 0, x))
    code = np.where(bad[..., None], 0x7f, code)
    return code.astype(np.uint8).reshape(*code.shape[:-2], -1), np.where(bad, 255, s + 127).astype(np.uint8)


def values(codes, scales, cols):
    v = np.concatenate([LEVELS, [np.nan], -LEVELS, [np.nan]])[codes].reshape(*scales.shape, 128)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v * s[..., None]).reshape(*scales.shape[:-1], -1)[..., :cols]


def rounded(x):
    return values(*quantise(x), np.shape(x)[-1])


def between(got, x, near):
    """Whether values `got` are what numbers within a factor 1 +- near of x [..., cols] stand
    for: between what the smaller and the larger ones do, for either's scale."""
    ends = [values(*quantise(x * f), x.shape[-1]) for f in (1 - near, 1 + near)]
    scale = [np.repeat(quantise(x * f)[1].astype(np.float64), 128, -1)[..., :x.shape[-1]] for f in (1 - near, 1 + near)]
    step = np.where(scale[0] != scale[1], np.exp2(scale[1] - 127 - 9), 0)  # the larger scale's smallest number
    lo, hi = np.minimum(*ends), np.maximum(*ends)
    return (got >= lo - step) & (got <= hi + step)


def norm(x, weight, residual, eps):
    h = x if residual is None else x + residual
    y = h / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * weight, h


def rotate(x, cos, sin, rotary_dim, neighbours):
    """x [rows, heads, dim] by cos and sin [rows, pairs]."""
    half = rotary_dim // 2
    y = x.copy()
    first = slice(0, rotary_dim, 2) if neighbours else slice(0, half)
    second = slice(1, rotary_dim, 2) if neighbours else slice(half, rotary_dim)
    a, b, c, s = x[..., first], x[..., second], cos[:, None], sin[:, None]
    y[..., first], y[..., second] = a * c - b * s, b * c + a * s
    return y
