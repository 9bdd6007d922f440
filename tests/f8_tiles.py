"""Which form of the kernels a product in block-scaled 8-bit floating point takes, by the library's rules: a copy of
them for tests that mean to reach every form, which fail when the rules move a shape to another one."""

from __future__ import annotations

CUS = 256  # of the device


def _up(a, b):
    return -(-a // b)


def forward_tile(m, n_out, kind, fused):
    """(weight rows, activation rows) of a tile of f8_linear or the fused call; from 65 rows on."""
    assert m > 64
    wide = kind == "float32"
    tiles = [(256, 128 if wide else 256), (128, 128), (128, 64), (64, 64), (192, 256)]
    cost = [57, 46, 29, 19] if wide else [59, 30, 23, 16, 53]
    if fused:
        cost = cost[:4]
    rows = n_out * (2 if fused else 1)
    time = [_up(_up(rows, bn) * _up(m, bm), CUS) * c for (bn, bm), c in zip(tiles, cost)]
    return tiles[time.index(min(time))]


TERMS = {"bfloat16": 1, "float16": 2, "float32": 3}  # parts of a gradient
PAIRS = {"bfloat16": 2, "float16": 3, "float32": 6}  # products of its parts with those of x's values


def _plan(rows, parts, cols, tile_rows, steps):
    if parts * _up(rows, 256) * _up(cols, 256) >= CUS // 2:
        return "large"
    ranges = min(CUS // (parts * _up(rows, tile_rows) * _up(cols, 128)), steps // 4, 16)
    return "ranges" if ranges > 1 else "small"


def dx_form(m, n, k, kind, parts):
    return _plan(m, 1, k, 64, parts * TERMS[kind] * _up(n, 64))


def dw_form(m, n, k, kind, parts):
    return _plan(n, parts, k, 128, PAIRS[kind] * _up(m, 64))
