"""The 8-bit block operators from their definitions, in numpy (fp64 unless said).

scale  s = max(fp32(absmax / F), 2^-126) over the finite values of the block; with pow2 the
       smallest power of two p >= 2^-126 with absmax <= F p
code   the nearest 8-bit value (ties to even) to fp32(x * fp32(1 / s)); NaN and infinities: NaN
value  fp32(code * s)
"""

import numpy as np
import torch

FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
_BITS = {"e4m3": (3, -6), "e5m2": (2, -14)}  # mantissa bits, exponent of the smallest normal


def _f32(x):
    return np.asarray(x, np.float64).astype(np.float32).astype(np.float64)


def round8(q, fmt):
    bits, low = _BITS[fmt]
    q = np.asarray(q, np.float64)
    e = np.maximum(np.frexp(np.where(np.isfinite(q), q, 0.0))[1] - 1, low)
    step = np.exp2((e - bits).astype(np.float64))
    return np.clip(np.rint(q / step) * step, -FMAX[fmt], FMAX[fmt])


def midpoints(fmt):
    """Values halfway between neighbouring non-negative codes, largest first."""
    bits, low = _BITS[fmt]
    n = 1 << bits
    vals = [j * 2.0 ** (low - bits) for j in range(n)]
    e = low
    while True:
        for j in range(n):
            v = (1 + j / n) * 2.0 ** e
            if v > FMAX[fmt]:
                vals = np.array(sorted(vals))
                return ((vals[1:] + vals[:-1]) / 2)[::-1].astype(np.float32)
            vals.append(v)
        e += 1


def _full(scales, by, rows, cols):
    """The scale of every element."""
    j = np.arange(cols) // 128
    if by == "rows":
        return scales[j].T
    return scales[np.arange(rows) // 128][:, j]


def quantize(x, by, fmt, pow2):
    """(codes as fp64 values, rows x cols; scales as fp32 in the library's layout)."""
    x = x.double().numpy() if isinstance(x, torch.Tensor) else np.asarray(x, np.float64)
    rows, cols = x.shape
    kb, rb = -(-cols // 128), -(-rows // 128)
    mag = np.where(np.isfinite(x), np.abs(x), 0.0)
    pad = np.zeros((rb * 128, kb * 128))
    pad[:rows, :cols] = mag
    amax = pad.reshape(rb * 128, kb, 128).max(2)
    amax = amax.reshape(rb, 128, kb).max(1) if by == "tiles" else amax[:rows]
    if pow2:
        m, e = np.frexp(amax / FMAX[fmt])  # m in [1/2, 1): exact, F's own power apart
        p = np.where(m == 0.5, e - 1, e)
        p = np.where(np.ldexp(FMAX[fmt], p) < amax, p + 1, p)
        s = np.exp2(np.maximum(np.where(amax > 0, p, -126), -126).astype(np.float64))
    else:
        s = np.maximum(_f32(amax / FMAX[fmt]), 2.0 ** -126)
    scales = (s.T if by == "rows" else s).astype(np.float32)
    f = _full(scales.astype(np.float64), by, rows, cols)
    with np.errstate(invalid="ignore"):
        q = _f32(np.where(np.isfinite(x), x, 0.0) * _f32(1.0 / f))
    codes = round8(q, fmt)
    return np.where(np.isfinite(x), codes, np.nan), np.ascontiguousarray(scales)


def restore(codes, scales, by, dtype=np.float32):
    rows, cols = codes.shape
    f = _full(np.asarray(scales, np.float64), by, rows, cols)
    return (np.asarray(codes, np.float64) * f).astype(dtype)
