"""Float64 oracle of the 8-bit block-scaled format and the operators on it (NumPy).

Value of a code: sign * 2^(ex - bias) * (1 + fr) for ex > 0, sign * 2^(1 - bias) * fr for
ex = 0, with bias 7 / 3 fraction bits (e4m3; code 0x7f is NaN, no infinities) or bias 15 /
2 fraction bits (e5m2; ex = 31 holds infinity and NaN).  A block of 128 (square 128 x 128,
or row 1 x 128) shares the scale 2^e, e the least integer with amax <= top * 2^e over the
block's finite magnitudes, clamped to [-127, 127], and 0 for amax = 0.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 128
TOP = {"e4m3": 448.0, "e5m2": 57344.0}


def code_values(fmt: str) -> np.ndarray:
    """The 256 values of a format."""
    frac, bias = {"e4m3": (3, 7), "e5m2": (2, 15)}[fmt]
    out = np.empty(256)
    for code in range(256):
        ex, fr = (code & 127) >> frac, (code & ((1 << frac) - 1)) / (1 << frac)
        v = math.ldexp(fr, 1 - bias) if ex == 0 else math.ldexp(1 + fr, ex - bias)
        if fmt == "e4m3" and (code & 127) == 127:
            v = math.nan
        if fmt == "e5m2" and ex == 31:
            v = math.inf if fr == 0 else math.nan
        out[code] = -v if code & 128 else v
    return out


def encode(v: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest code of each (already scaled) value, ties to the even code."""
    pos = code_values(fmt)[:127 if fmt == "e4m3" else 124]     # finite, ascending
    a = np.abs(v)
    fin = np.where(np.isfinite(a), a, 0.0)
    hi = np.clip(np.searchsorted(pos, fin, side="left"), 1, len(pos) - 1)
    lo = hi - 1
    mid = 0.5 * (pos[lo] + pos[hi])
    c = np.where(fin > mid, hi, np.where(fin < mid, lo, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(np.isnan(v), 0x7f, np.where(np.isinf(v), 0x7f if fmt == "e4m3" else 0x7c, c))
    return (c | np.where(np.signbit(v) & ~np.isnan(v), 0x80, 0)).astype(np.uint8)


def exponent(amax: float, fmt: str) -> int:
    if amax == 0.0:
        return 0
    e = math.frexp(amax)[1] - (9 if fmt == "e4m3" else 16)     # top = 0.875 * 2^9 or 2^16
    while amax > math.ldexp(TOP[fmt], e):
        e += 1
    while amax <= math.ldexp(TOP[fmt], e - 1):
        e -= 1
    return max(-127, min(127, e))


def expand(e: np.ndarray, rows: int, cols: int, blocks: str) -> np.ndarray:
    """Block exponents to one per entry."""
    full = np.repeat(e, BLOCK, axis=1)[:, :cols]
    return np.repeat(full, BLOCK, axis=0)[:rows] if blocks == "square" else full


def quantize(x: np.ndarray, fmt: str = "e4m3", blocks: str = "square"):
    """(codes [rows, cols], exponents [row blocks or rows, column blocks])."""
    x = np.asarray(x, dtype=np.float64)
    r, c = x.shape
    step = BLOCK if blocks == "square" else 1
    e = np.zeros((-(-r // step), -(-c // BLOCK)), dtype=np.int64)
    codes = np.zeros((r, c), dtype=np.uint8)
    for i in range(e.shape[0]):
        for j in range(e.shape[1]):
            blk = x[i * step:(i + 1) * step, j * BLOCK:(j + 1) * BLOCK]
            fin = np.abs(blk[np.isfinite(blk)])
            e[i, j] = exponent(float(fin.max()) if fin.size else 0.0, fmt)
            codes[i * step:(i + 1) * step, j * BLOCK:(j + 1) * BLOCK] = encode(np.ldexp(blk, int(-e[i, j])), fmt)
    return codes, e


def dequantize(codes: np.ndarray, e: np.ndarray, fmt: str = "e4m3", blocks: str = "square") -> np.ndarray:
    r, c = codes.shape
    return code_values(fmt)[codes] * np.exp2(expand(e, r, c, blocks).astype(np.float64))


def relu2(u: np.ndarray) -> np.ndarray:
    return np.where(np.isnan(u), u, np.square(np.maximum(u, 0.0)))


def relu2_backward(dy: np.ndarray, h: np.ndarray) -> np.ndarray:
    """dy * d(relu(u)^2)/du from h = relu(u)^2: the slope is 2 relu(u) = 2 sqrt(h)."""
    return 2.0 * np.sqrt(h) * dy


def matmul(a: np.ndarray, b: np.ndarray, c=None, epilogue: str = "none", saved=None):
    """(result, bound): epilogue(c + a @ b) in float64 and sum |a||b| + |c| per entry, the
    scale that float32 accumulation errors are relative to (before the epilogue)."""
    with np.errstate(invalid="ignore"):
        d = a @ b
        mag = np.abs(a) @ np.abs(b)
    if c is not None:
        d = d + c
        mag = mag + np.abs(c)
    if epilogue == "relu2":
        d = relu2(d)
    elif epilogue == "relu2_backward":
        d = relu2_backward(d, saved)
    return d, mag
