"""Float64 oracle of the 8-bit operands and their products (numpy, test infrastructure).

An element is value8 * 2^e, one e per 128 columns of a row, e the least integer
>= -126 with the block's largest finite magnitude <= 1.75 * 2^(t + e) (t = 8 for e4m3,
15 for e5m2), 0 for a block of zeros. Values are rounded to the nearest 8-bit number,
ties to even.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
# format: exponent bits, mantissa bits, bias, exponent of the largest value
FORMATS = {"e4m3": (4, 3, 7, 8), "e5m2": (5, 2, 15, 15)}


def up(n: int, to: int) -> int:
    return -(-n // to) * to


def decode_table(fmt: str) -> np.ndarray:
    """The 256 values of a format (e4m3: no infinities, 0x7f and 0xff NaN; e5m2 as IEEE)."""
    ebits, mbits, bias, _ = FORMATS[fmt]
    out = np.zeros(256)
    for b in range(256):
        sign = -1.0 if b & 0x80 else 1.0
        e = (b >> mbits) & ((1 << ebits) - 1)
        m = b & ((1 << mbits) - 1)
        if fmt == "e4m3" and (b & 0x7f) == 0x7f:
            v = np.nan
        elif fmt == "e5m2" and e == (1 << ebits) - 1:
            v = np.inf if m == 0 else np.nan
        elif e == 0:
            v = m * 2.0 ** (1 - bias - mbits)
        else:
            v = (1.0 + m * 2.0 ** -mbits) * 2.0 ** (e - bias)
        out[b] = sign * v
    return out


def round_to(x: np.ndarray, fmt: str) -> np.ndarray:
    """Nearest values of the format, ties to even; |x| <= 1.75 * 2^t, infinities and NaN
    as the format has them."""
    _, mbits, bias, _ = FORMATS[fmt]
    with np.errstate(all="ignore"):
        _, ex = np.frexp(np.where(np.isfinite(x), x, 0.0))
        step = 2.0 ** (np.maximum(ex - 1, 1 - bias) - mbits)
        y = np.rint(x / step) * step
    if fmt == "e4m3":
        y = np.where(np.isfinite(x), y, np.nan)
    else:
        y = np.where(np.isfinite(x), y, x)
    return y


def block_exponent(amax: np.ndarray, fmt: str) -> np.ndarray:
    half, ex = np.frexp(amax)               # amax = half * 2^ex, half in [0.5, 1)
    e = ex - 1 - FORMATS[fmt][3] + (half > 0.875)
    return np.where(amax > 0, np.maximum(e, -126), 0).astype(np.int64)


def quantize(x: np.ndarray, fmt: str, blocks: bool = False):
    """(values [rows, cols padded], exponents [rows, blocks]) of a 2-D matrix."""
    rows, cols = x.shape
    wide = np.zeros((up(rows, BLOCK) if blocks else rows, up(cols, BLOCK)))
    wide[:rows, :cols] = x
    b = wide.reshape(-1, BLOCK if blocks else 1, wide.shape[1] // BLOCK, BLOCK)
    mag = np.where(np.isfinite(b), np.abs(b), 0.0)
    e = block_exponent(mag.max(axis=(1, 3), initial=0.0, keepdims=True), fmt)
    q = round_to(b * 2.0 ** -e.astype(np.float64), fmt).reshape(wide.shape)[:rows]
    e = np.broadcast_to(e[..., 0], b.shape[:3]).reshape(-1, wide.shape[1] // BLOCK)[:rows]
    return q, e


def gather(x: np.ndarray, index, div: int, weight=None) -> np.ndarray:
    """Rows index // div of x (float32 products with weight[index]), zeros outside."""
    out = np.zeros((len(index), x.shape[1]))
    for r, i in enumerate(index):
        if i < 0 or i // div >= len(x) or (weight is not None and i >= len(weight)):
            continue
        row = x[i // div]
        out[r] = row if weight is None else (row.astype(np.float32) * np.float32(weight[i])).astype(np.float64)
    return out


def dequantize(q: np.ndarray, e: np.ndarray, cols: int) -> np.ndarray:
    return (q * 2.0 ** np.repeat(e, BLOCK, axis=1).astype(np.float64))[:, :cols]
