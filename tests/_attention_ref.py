"""Plain forms, in 64 bits, of the 8-bit operands, the head norm with rotation and the paged 8-bit cache.

The steps that a definition takes in 32 bits (a scale, its inverse, the scaled value behind a
code) are rounded to 32 bits here as well, so that codes and scales can be compared bit for bit.
"""
from __future__ import annotations

import numpy as np

ROW_FLOOR = np.float32(2.0 ** -100)
PAGE_FLOOR = np.float32(2.0 ** -64)


def scale_of(amax, floor):
    """Scale of values with the largest magnitude amax (fp32)."""
    with np.errstate(all="ignore"):
        s = np.maximum((np.asarray(amax, np.float32) / np.float32(127)).astype(np.float32), floor)
    return np.where(np.isfinite(amax), s, np.float32(np.nan)).astype(np.float32)


def codes_of(x, s):
    """Codes of x (fp32) under scales s that broadcast against it."""
    with np.errstate(all="ignore"):
        r = np.where(np.isnan(s), np.float32(0), np.float32(1) / s).astype(np.float32)
        y = np.rint((x * r).astype(np.float32))
    return np.where(np.isnan(y), 0, np.clip(y, -127, 127)).astype(np.int8)


def s8_quantize(X):
    X = np.asarray(X, np.float32)
    rows, K = X.shape
    finite = np.isfinite(X).all(axis=1)
    amax = np.where(finite, np.abs(np.where(np.isfinite(X), X, 0)).max(axis=1), np.float32(np.inf))
    s = scale_of(amax, ROW_FLOOR)
    q = np.zeros((rows, -(-K // 16) * 16), np.int8)
    q[:, :K] = codes_of(X, s[:, None])
    return q, s


def turn(x, cos, sin, R, style):
    """The rotation of the first R values of x (T x H x D) by cos, sin (T x R / 2)."""
    y = np.array(x, dtype=np.float64)
    i = np.arange(R // 2)
    a, b = (i, i + R // 2) if style == "half" else (2 * i, 2 * i + 1)
    c, s = cos[:, None, :], sin[:, None, :]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def turn_size(x, cos, sin, R, style):
    """The sum of the magnitudes that the rotation adds up."""
    y = np.abs(np.array(x, dtype=np.float64))
    x = y.copy()
    i = np.arange(R // 2)
    a, b = (i, i + R // 2) if style == "half" else (2 * i, 2 * i + 1)
    c, s = np.abs(cos)[:, None, :], np.abs(sin)[:, None, :]
    y[..., a] = x[..., a] * c + x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def rms(x, eps):
    return 1 / np.sqrt((x * x).mean(axis=2) + eps)


class Cache:
    """A cache as numpy arrays, with the plain append and read."""

    def __init__(self, kq, vq, ks, vs):
        self.q = {"k": np.array(kq), "v": np.array(vq)}
        self.s = {"k": np.array(ks), "v": np.array(vs)}
        self.pages, self.heads, self.page, self.D = self.q["k"].shape

    def append(self, which, X, table, starts, lengths):
        q, s, page = self.q[which], self.s[which], self.page
        X = np.asarray(X, np.float32)
        for b in range(len(lengths)):
            r0, n = int(starts[b]), int(starts[b + 1] - starts[b])
            lo, hi = max(0, int(lengths[b]) - n), min(int(lengths[b]), table.shape[1] * page)
            first = int(lengths[b]) - n
            for j in range(lo // page, -(-hi // page)) if n > 0 and hi > lo else ():
                p = int(table[b][j])
                if not 0 <= p < self.pages:
                    continue
                a, z = max(lo, j * page), min(hi, (j + 1) * page)
                kept = a - j * page
                x = X[r0 + a - first:r0 + z - first]
                for h in range(self.heads):
                    v = x[:, h]
                    amax = np.abs(v).max() if np.isfinite(v).all() else np.float32(np.inf)
                    now = scale_of(amax, PAGE_FLOOR)
                    if kept:
                        old = s[p, h]
                        if np.isnan(old) or old > now:
                            now = old
                        if not old == now:
                            with np.errstate(all="ignore"):
                                f = np.float32(old / now)
                                y = np.rint((q[p, h, :kept].astype(np.float32) * f).astype(np.float32))
                            q[p, h, :kept] = np.where(np.isnan(y), 0, y).astype(np.int8)
                    s[p, h] = now
                    q[p, h, kept:kept + z - a] = codes_of(v, now)

    def tokens(self, which, table, b, n):
        """The first n tokens of sequence b as values and as scales (n x heads x D, n x heads)."""
        v = np.full((n, self.heads, self.D), np.nan)
        sc = np.full((n, self.heads), np.nan)
        for j in range(n):
            col = j // self.page
            p = int(table[b][col]) if col < table.shape[1] else -1
            if 0 <= p < self.pages:
                sc[j] = self.s[which][p].astype(np.float64)
                v[j] = self.q[which][p, :, j % self.page].astype(np.float64) * sc[j][:, None]
        return v, sc
