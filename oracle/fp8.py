"""Plain CPU oracle of the 8-bit storage, its products and the norm (numpy, fp64).

Codes are OCP 8-bit floats in blocks of 128 columns of one row (block_rows = 1)
or of 128 rows (block_rows = 128), one fp32 scale per block:

    amax = max(max |x|, 2^-100), scale = fl32(amax / F),
    code = nearest 8-bit value to fl32(x * fl32(F * fl32(1 / amax))), ties to even.

A NaN keeps its sign-less NaN code and does not count for its block's amax.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
FLOOR = np.float32(2.0 ** -100)
FORMATS = {"e4m3": (3, 7, 448.0), "e5m2": (2, 15, 57344.0)}  # mantissa bits, exponent bias, largest value


def code_values(fmt: str) -> np.ndarray:
    """fp64 [256]: the value of every code."""
    man, bias, largest = FORMATS[fmt]
    out = np.empty(256, np.float64)
    for c in range(256):
        sign = -1.0 if c & 0x80 else 1.0
        e, m = (c & 0x7F) >> man, c & ((1 << man) - 1)
        v = m * 2.0 ** (1 - bias - man) if e == 0 else (1.0 + m / (1 << man)) * 2.0 ** (e - bias)
        if fmt == "e4m3":
            v = np.nan if (c & 0x7F) == 0x7F else v
        elif e == 31:
            v = np.nan if m else np.inf
        out[c] = sign * v
    return out


def encode(x: np.ndarray, fmt: str) -> np.ndarray:
    """uint8 codes of finite or NaN values with |x| <= the largest value (plus less than half a step): the nearest
    code, the even one on a tie; a NaN becomes the positive NaN code with all mantissa bits set."""
    vals = code_values(fmt)
    pos = vals[:128]
    n = int(np.sum(np.isfinite(pos)))
    grid = pos[:n]  # ascending
    a = np.abs(np.asarray(x, np.float64))
    a = np.where(np.isnan(a), 0.0, a)
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")   # codes whose upper midpoint is below a
    tie = (lo < n - 1) & (a == mid[np.minimum(lo, n - 2)])
    code = np.where(tie & (lo % 2 == 1), lo + 1, lo).astype(np.uint8)
    code = code | (np.signbit(x).astype(np.uint8) << 7)
    return np.where(np.isnan(x), np.uint8(0x7F), code).astype(np.uint8)


def _spread(b: np.ndarray, block_rows: int, rows: int, cols: int) -> np.ndarray:
    return np.repeat(np.repeat(b, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]


def block_scales(x: np.ndarray, block_rows: int, fmt: str):
    """(scale, multiplier) fp32 per block of a fp32 [rows][cols]."""
    rows, cols = x.shape
    F = np.float32(FORMATS[fmt][2])
    rb, cb = -(-rows // block_rows), -(-cols // BLOCK)
    amax = np.zeros((rb, cb), np.float32)
    for i in range(rb):
        for j in range(cb):
            b = np.abs(x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK])
            b = b[~np.isnan(b)]
            amax[i, j] = b.max() if b.size else 0.0
    amax = np.maximum(amax, FLOOR)
    with np.errstate(over="ignore"):
        return (amax / F).astype(np.float32), F * (np.float32(1.0) / amax)


def quantize(x: np.ndarray, block_rows: int, fmt: str):
    """(codes uint8 [rows][cols], scales fp32)."""
    x = np.asarray(x, np.float32)
    scale, mul = block_scales(x, block_rows, fmt)
    with np.errstate(invalid="ignore"):
        v = x * _spread(mul, block_rows, *x.shape)
    return encode(v, fmt), scale


def dequantize(codes: np.ndarray, scales: np.ndarray, block_rows: int, fmt: str) -> np.ndarray:
    """fp32 [rows][cols] = fl32(code * scale)."""
    v = code_values(fmt)[codes].astype(np.float32)
    with np.errstate(invalid="ignore"):
        return v * _spread(np.asarray(scales, np.float32), block_rows, *codes.shape)


def matmul(a, a_scales, a_fmt, w, w_scales, transpose=False, A2=None, B2=None):
    """(C, S, Q) in fp64: the product of the dequantized values, the sum of its terms' magnitudes, and the square root
    of the sum of their squares."""
    A = code_values(a_fmt)[a] * _spread(np.asarray(a_scales, np.float64), 1, *a.shape)
    W = code_values("e4m3")[w] * _spread(np.asarray(w_scales, np.float64), BLOCK, *w.shape)
    B = W if transpose else W.T
    C, S, Q = A @ B, np.abs(A) @ np.abs(B), (A * A) @ (B * B)
    if A2 is not None:
        A2, B2 = np.asarray(A2, np.float64), np.asarray(B2, np.float64)
        C, S, Q = C + A2 @ B2.T, S + np.abs(A2) @ np.abs(B2).T, Q + (A2 * A2) @ (B2 * B2).T
    return C, S, np.sqrt(Q)


def rmsnorm(h, w, eps):
    """(y, rstd) in fp64 of h [M][H] (the residual already added and rounded)."""
    h, w = np.asarray(h, np.float64), np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, 1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_grad(dy, h, w, rstd, dh=None):
    """(dx, dw) in fp64."""
    dy, h, w = (np.asarray(t, np.float64) for t in (dy, h, w))
    xhat = h * np.asarray(rstd, np.float64)[:, None]
    u = dy * w
    dx = np.asarray(rstd, np.float64)[:, None] * (u - xhat * np.mean(u * xhat, 1, keepdims=True))
    return (dx if dh is None else dx + np.asarray(dh, np.float64)), np.sum(dy * xhat, 0)
