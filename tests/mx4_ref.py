"""The microscaled 4-bit format and its operators in float64 numpy, from their definition."""
import numpy as np

LEVELS = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
MIDDLES = (LEVELS[1:] + LEVELS[:-1]) / 2


def quantise(x):
    """x [..., cols] -> codes uint8 [..., cols up to 32], scale bytes [..., blocks]."""
    x = np.asarray(x, np.float64)
    pad = -x.shape[-1] % 32
    x = np.concatenate([x, np.zeros((*x.shape[:-1], pad))], -1)
    x = x.reshape(*x.shape[:-1], x.shape[-1] // 32, 32)
    top = np.abs(x).max(-1)
    bad = ~np.isfinite(top)
    s = np.zeros(top.shape, np.int64)
    ok = ~bad & (top > 0)
    s[ok] = np.clip(np.frexp(top[ok])[1] - 3, -125, 125)
    a = np.abs(np.where(bad[..., None], 0, x)) * np.ldexp(1.0, -s)[..., None]
    lo = np.searchsorted(MIDDLES, a, side="left")    # a tie goes down
    hi = np.searchsorted(MIDDLES, a, side="right")   # a tie goes up
    code = np.where(lo % 2 == 0, lo, hi)
    code = np.where(lo == hi, lo, code) + 8 * np.signbit(np.where(bad[..., None], 0, x))
    return code.astype(np.uint8).reshape(*code.shape[:-2], code.shape[-2] * 32), np.where(bad, 255, s + 127).astype(np.uint8)


def values(codes, scales, cols):
    v = np.concatenate([LEVELS, -LEVELS])[codes].reshape(*scales.shape, 32)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v * s[..., None]).reshape(*scales.shape[:-1], scales.shape[-1] * 32)[..., :cols]


def rounded(x):
    return values(*quantise(x), np.shape(x)[-1])


def unpack(codes):
    codes = np.asarray(codes)
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)


def attend_rows(q, positions, k, v, there, scale, window, sinks):
    """q [n, Hq, D] at `positions`; k, v [T, Hkv, D]; there [T]: the token has a page.
    Gives o and, for tolerances, sum p |v| and the largest sum |q k| of each row."""
    n, hq, d = q.shape
    group = hq // k.shape[1]
    o, mag, dot = (np.zeros((n, hq, d)) for _ in range(3))
    t = np.arange(k.shape[0])
    for i in range(n):
        seen = there & (t <= positions[i])
        if window:
            seen &= (t > positions[i] - window) | (t < sinks)
        if not seen.any():
            continue
        for h in range(hq):
            kk, vv = k[seen, h // group], v[seen, h // group]
            z = kk @ q[i, h] * scale
            with np.errstate(invalid="ignore"):
                p = np.exp(z - z.max())
                p /= p.sum()
                o[i, h] = p @ vv
                mag[i, h] = p @ np.abs(vv)
            dot[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
    return o, mag, dot
