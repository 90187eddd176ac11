"""Plain forms, in numpy and 64 bits, of the microscaled 4-bit operators and layer norm.

The steps that the quantizer's definition takes in 32 bits (the quotient behind a
block scale, the scaled value behind a code) are rounded to 32 bits here as well,
so codes and scale bytes can be compared bit for bit.
"""
from __future__ import annotations

import numpy as np

BLOCK = {"nv": 16, "mx": 32}
GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)
E4M3 = np.array([(m / 8 * 2.0 ** -6) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127], dtype=np.float64)  # 127 is NaN


def _nearest_even(a, grid):
    """Index of the grid value nearest to a >= 0; ties to the even index; above the grid: its end."""
    hi = np.searchsorted(grid, a, side="left").clip(0, len(grid) - 1)
    lo = (hi - 1).clip(0)
    mid = (grid[lo] + grid[hi]) / 2
    up = (a > mid) | ((a == mid) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def codes_and_bytes(X, fmt, ts=1.0):
    """X (rows x K, finite or not) -> codes (rows x K up to whole blocks, values 0..15), scale bytes."""
    b = BLOCK[fmt]
    X = np.asarray(X, dtype=np.float32)
    rows, K = X.shape
    nb = -(-K // b)
    x = np.zeros((rows, nb * b), dtype=np.float32)
    x[:, :K] = X
    x = x.reshape(rows, nb, b)
    bad = ~np.isfinite(x).all(axis=2)
    amax = np.where(bad, 0, np.abs(np.where(np.isfinite(x), x, 0)).max(axis=2)).astype(np.float32)
    with np.errstate(all="ignore"):
        if fmt == "nv":
            ts = np.float32(ts)
            q = (amax / (np.float32(6) * ts)).astype(np.float32)
            byte = _nearest_even(q.astype(np.float64), E4M3)
            d = (E4M3[byte].astype(np.float32) * ts).astype(np.float32)
            r = np.where(byte > 0, np.float32(1) / d, np.float32(0)).astype(np.float32)
            byte = np.where(bad, 0x7F, byte)
        else:
            e = np.where(amax > 0, np.floor(np.log2(np.maximum(amax, 1e-45).astype(np.float64))), -200) - 2
            e = np.clip(e, -127, 127)
            byte = np.where(bad, 0xFF, e + 127).astype(np.int64)
            r = np.exp2(-e).astype(np.float32)
        y = (x * r[:, :, None]).astype(np.float32)
    y = np.where(np.isfinite(y), y, 0)
    code = _nearest_even(np.abs(y).astype(np.float64), GRID) | np.where(np.signbit(y), 8, 0)
    return code.reshape(rows, -1).astype(np.uint8), byte.astype(np.uint8)


def scale_values(byte, fmt):
    byte = np.asarray(byte).astype(np.int64)
    if fmt == "nv":
        return np.where(byte == 127, np.nan, E4M3[np.minimum(byte, 126)])
    return np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))


def code_values(code):
    return np.where(code & 8, -1.0, 1.0) * GRID[code & 7]


def values(code, byte, fmt, K):
    """Codes times block scales in 64 bits, without the tensor scale."""
    b = BLOCK[fmt]
    v = code_values(code).reshape(code.shape[0], -1, b) * scale_values(byte, fmt)[:, :, None]
    return v.reshape(code.shape[0], -1)[:, :K]


def pack(code, byte):
    """The packed layout, element by element: (codes, scales), zero behind the edges."""
    rows, n = code.shape
    nb = byte.shape[1]
    q = np.zeros((rows, -(-n // 32) * 32), dtype=np.uint8)
    q[:, :n] = code
    q = q[:, 0::2] | (q[:, 1::2] << 4)
    tr, tc = -(-rows // 128), -(-nb // 4)
    s = np.zeros((tr, tc, 512), dtype=np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    s[r // 128, c // 4, 16 * (r % 32) + 4 * (r % 128 // 32) + c % 4] = byte
    return q, s


def quantized(X, fmt, ts=1.0):
    """What X's packed form stands for, without the tensor scale."""
    code, byte = codes_and_bytes(X, fmt, ts)
    return values(code, byte, fmt, np.asarray(X).shape[1])


def layer_norm(X, gamma, beta, eps):
    X = np.asarray(X, dtype=np.float64)
    mean = X.mean(axis=1, keepdims=True)
    rstd = 1 / np.sqrt(((X - mean) ** 2).mean(axis=1, keepdims=True) + eps)
    y = (X - mean) * rstd
    if gamma is not None:
        y = y * np.asarray(gamma, dtype=np.float64)
    if beta is not None:
        y = y + np.asarray(beta, dtype=np.float64)
    return y, mean[:, 0], rstd[:, 0]


def layer_norm_backward(dY, X, gamma, eps):
    dY, X = np.asarray(dY, dtype=np.float64), np.asarray(X, dtype=np.float64)
    _, mean, rstd = layer_norm(X, None, None, eps)
    xh = (X - mean[:, None]) * rstd[:, None]
    d = dY if gamma is None else dY * np.asarray(gamma, dtype=np.float64)
    dx = rstd[:, None] * (d - d.mean(axis=1, keepdims=True) - xh * (d * xh).mean(axis=1, keepdims=True))
    return dx, (dY * xh).sum(axis=0), dY.sum(axis=0)
