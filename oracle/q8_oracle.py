"""Plain oracle of the 8-bit operators: E4M3 codes with a scale per block.

numpy, fp64; scales are rounded once to fp32.  Shares nothing with the kernels.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
TOP = 448.0
FLOOR = 2.0 ** -120


def _table():
    t = np.zeros(256)
    for b in range(256):
        sign, e, m = -1.0 if b & 128 else 1.0, (b >> 3) & 15, b & 7
        if e == 15 and m == 7:
            t[b] = np.nan
        elif e == 0:
            t[b] = sign * m * 2.0 ** -9
        else:
            t[b] = sign * (8 + m) * 2.0 ** (e - 10)
    return t


E4M3 = _table()
_POS = E4M3[:127]                       # 0 .. 448, ascending


def decode(codes):
    return E4M3[np.asarray(codes, dtype=np.uint8)]


def encode(v):
    """Codes of |v| <= 448 (and NaN), to nearest, ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.abs(np.nan_to_num(v, nan=0.0))
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= _POS[126], 126, code)
    code = np.where(np.signbit(v), code | 128, code)
    return np.where(np.isnan(v), 0x7f, code).astype(np.uint8)


def e8m0(byte):
    b = np.asarray(byte, dtype=np.int64)
    return np.where(b == 255, np.nan, 2.0 ** (b - 127.0))


def nblk(n):
    return -(-n // BLOCK)


def spread(scales, block_rows, rows, cols):
    """One scale per element."""
    s = np.repeat(np.asarray(scales, dtype=np.float64), block_rows, axis=0)[:rows]
    return np.repeat(s, BLOCK, axis=1)[:, :cols]


def dequantize(codes, scales, block_rows=1):
    with np.errstate(invalid="ignore"):
        return decode(codes) * spread(scales, block_rows, *codes.shape)


def block_max(x, block_rows):
    rows, cols = x.shape
    out = np.zeros((-(-rows // block_rows), nblk(cols)), dtype=x.dtype)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = np.max(np.abs(x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]))
    return out


def scale_of(amax, kind):
    """fp32 scales of fp32 maxima (NaN where a block is not finite)."""
    with np.errstate(invalid="ignore", over="ignore"):
        s = np.maximum(amax.astype(np.float32) / np.float32(TOP), np.float32(FLOOR))
        if kind == "e8m0":
            m, e = np.frexp(s.astype(np.float64))
            s = np.exp2(np.where(m == 0.5, e - 1, e)).astype(np.float32)
        return np.where(np.isfinite(amax), s, np.float32(np.nan)).astype(np.float32)


def quotients(x, block_rows=1, kind="f32"):
    """x over its block's scale (before the scale's rounding), in fp64, and
    the fp32 scales."""
    x = np.asarray(x, dtype=np.float32)
    amax = block_max(x, block_rows)
    s = scale_of(amax, kind)
    with np.errstate(invalid="ignore", over="ignore"):
        d = s.astype(np.float64) if kind == "e8m0" else np.maximum(amax.astype(np.float64) / TOP, FLOOR)
        d = np.where(np.isnan(s), np.nan, d)
        return x.astype(np.float64) / spread(d, block_rows, *x.shape), s


def quantize(x, block_rows=1, kind="f32"):
    """Codes and scales (as fp32 values) of fp32 values, by the coding rule."""
    v, s = quotients(x, block_rows, kind)
    return encode(v), s


def rmsnorm(x, residual=None, gamma=None, eps=1e-6):
    """(normed, h, rstd, h * rstd) in fp64."""
    h = np.asarray(x, dtype=np.float64)
    if residual is not None:
        h = h + np.asarray(residual, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
        xn = h * r[:, None]
        return (xn if gamma is None else xn * np.asarray(gamma, dtype=np.float64)), h, r, xn


def rmsnorm_vjp(xn, rstd, dn, gamma=None, dres=None):
    """(dh, dgamma) from the normed rows h * rstd."""
    u = dn if gamma is None else dn * gamma
    dh = rstd[:, None] * (u - xn * np.mean(u * xn, axis=1, keepdims=True))
    return dh if dres is None else dres + dh, np.sum(dn * xn, axis=0)


def matmul(a_codes, a_scales, w_codes, w_scales):
    return dequantize(a_codes, a_scales, 1) @ dequantize(w_codes, w_scales, BLOCK).T


def wgrad(dy, x_codes, x_scales):
    return np.asarray(dy, dtype=np.float64).T @ dequantize(x_codes, x_scales, 1)
