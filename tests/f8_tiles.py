"""Which form of the kernels a product in block-scaled 8-bit floating point takes, by the library's rules: a copy of
them for tests that mean to reach every form, which fail when the rules move a shape to another one."""

from __future__ import annotations

CUS = 256  # of the device


def _up(a, b):
    return -(-a // b)


WEIGHT_ROWS, ROWS = (256, 128, 128, 64, 192), {"wide": (128, 128, 64, 64, 256), "narrow": (256, 128, 64, 64, 256)}
COST = {"wide": (57, 46, 29, 19, 53), "narrow": (59, 30, 23, 16, 53)}  # of a round, by the width of the results


def forward_tile(m, n_out, kind, fused):
    """(weight rows, activation rows) of a tile of f8_linear or the fused call; from 65 rows on."""
    assert m > 64
    width = "wide" if kind == "float32" else "narrow"
    tiles = list(zip(WEIGHT_ROWS, ROWS[width]))
    if fused or width == "wide":
        tiles = tiles[:4]
    rows = n_out * (2 if fused else 1)
    time = [_up(_up(rows, bn) * _up(m, bm), CUS) * c for (bn, bm), c in zip(tiles, COST[width])]
    return tiles[time.index(min(time))]


TERMS = {"bfloat16": 1, "float16": 2, "float32": 3}  # parts of a gradient
PAIRS = {"bfloat16": 2, "float16": 3, "float32": 6}  # products of its parts with those of x's values


def _plan(rows, parts, cols, tile_rows, steps):
    """(form, ranges that the sum is cut into)"""
    if parts * _up(rows, 256) * _up(cols, 256) >= CUS // 2:
        return "large", 1
    ranges = min(CUS // (parts * _up(rows, tile_rows) * _up(cols, 128)), steps // 4, 16)
    return ("ranges", ranges) if ranges > 1 else ("small", 1)


def _dx(m, n, k, kind, parts):
    return _plan(m, 1, k, 64, parts * TERMS[kind] * _up(n, 64))


def _dw(m, n, k, kind, parts):
    return _plan(n, parts, k, 128, PAIRS[kind] * _up(m, 64))


def dx_form(*sizes):
    return _dx(*sizes)[0]


def dw_form(*sizes):
    return _dw(*sizes)[0]


def backward_bytes(m, n, k, kind, parts):
    """The workspace that these forms need: parts of the gradients and of x's values, and the ranges' sums."""
    of_dx, of_dw = _dx(m, n, k, kind, parts)[1], _dw(m, n, k, kind, parts)[1]
    value_terms = 3 if kind == "float32" else 2
    pieces = (2 * TERMS[kind] * m * parts * 64 * _up(n, 64), 2 * value_terms * 64 * _up(m, 64) * k,
              4 * of_dx * m * k if of_dx > 1 else 0, 4 * of_dw * parts * n * k if of_dw > 1 else 0)
    return sum(256 * _up(p, 256) for p in pieces)
