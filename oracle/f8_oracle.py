"""Float64 reference of the block-scaled 8-bit floating-point linears (numpy, CPU).

Codes are OCP e4m3 bytes; value = code * scale with one float32 scale for every 128 inputs of
an activation row and for every 128 x 128 block of a weight matrix."""

from __future__ import annotations

import numpy as np

F8_BLOCK = 128
F8_TOP = 448.0
F8_TINY = 2.0 ** -116


def e4m3_table():
    """The 256 codes' values in float64: sign, 4 bits of exponent (bias 7), 3 of fraction; 0x7F and 0xFF NaN."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        mag = f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        if c & 127 == 127:
            mag = np.nan
        v[c] = -mag if c & 128 else mag
    return v


def e4m3_encode(v):
    """Codes nearest to float64 values of magnitude at most 448, ties to the even code."""
    v = np.asarray(v, dtype=np.float64)
    mags = e4m3_table()[:127]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(mags, a), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - mags[lo], mags[hi] - a
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    return np.where(np.signbit(v), code | 128, code).astype(np.uint8)


def _block_tops(x, rows):
    n, k = x.shape
    nb, kb = -(-n // rows), -(-k // F8_BLOCK)
    whole = np.zeros((nb * rows, kb * F8_BLOCK))
    whole[:n, :k] = np.abs(x)
    return whole.reshape(nb, rows, kb, F8_BLOCK).max(axis=(1, 3))  # a NaN stays one


def f8_quantize_ref(x, rows, pow2):
    """(codes uint8 [n][k], scales float32) of blocks of `rows` rows x 128 columns; x holds float32 values."""
    x = np.asarray(x, dtype=np.float64)
    n, k = x.shape
    top = _block_tops(x, rows)
    bad, live = ~np.isfinite(top), np.isfinite(top) & (top >= F8_TINY)
    safe = np.where(live, top, F8_TOP)
    if pow2:
        power = np.floor(np.log2(safe / F8_TOP))
        power = np.where(2.0 ** power * F8_TOP < safe, power + 1, power)
        scale = 2.0 ** power
        by = 1.0 / scale
    else:
        scale = (safe / F8_TOP).astype(np.float32)
        by = (F8_TOP / safe).astype(np.float32).astype(np.float64)
    scale = np.where(live, scale, np.where(bad, np.nan, 0.0)).astype(np.float32)
    by = np.where(live, by, 0.0)
    spread = np.repeat(np.repeat(by, rows, axis=0)[:n], F8_BLOCK, axis=1)[:, :k]
    dead = np.repeat(np.repeat(bad, rows, axis=0)[:n], F8_BLOCK, axis=1)[:, :k]
    with np.errstate(over="ignore", invalid="ignore"):
        v = (np.where(dead, 0.0, x) * spread).astype(np.float32).astype(np.float64)
    code = e4m3_encode(np.clip(v, -F8_TOP, F8_TOP))
    return np.where(dead, np.uint8(0x7F), code).astype(np.uint8), scale


def f8_values(codes, scales, rows):
    """The float64 values [n][k] that codes and scales of blocks of `rows` rows stand for."""
    n, k = codes.shape
    s = np.repeat(np.repeat(np.asarray(scales, np.float64), rows, axis=0)[:n], F8_BLOCK, axis=1)[:, :k]
    return e4m3_table()[codes] * s


def f8_weight_values(codes, scales, parts=1):
    """f8_values of a matrix of `parts` equal parts with blocks of their own."""
    n = codes.shape[0] // parts
    nb = -(-n // F8_BLOCK)
    return np.concatenate([f8_values(codes[p * n:(p + 1) * n], scales[p * nb:(p + 1) * nb], F8_BLOCK)
                           for p in range(parts)])


def _sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def f8_gate_up_ref(gu):
    """SiLU(g) * u of products beside each other."""
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    return g * _sigmoid(g) * u


def f8_gate_up_gradient_ref(gu, dh):
    """[dg du] of SiLU(g) * u."""
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    s = _sigmoid(g)
    return np.concatenate([dh * u * s * (1 + g * (1 - s)), dh * g * s], axis=1)
