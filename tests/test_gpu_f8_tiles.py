"""Every tile of the 8-bit floating-point products and gradients on general operands: scales of their own, several
whole blocks of inputs and a cut one, rows and outputs that end inside a tile.  Limits as in f8_cases.py and the tests
of the small forms; which tile a shape takes is asserted, so that a rule that moves shapes leaves none untested."""

from __future__ import annotations

import numpy as np
import pytest

from f8_cases import TYPES, as_type, check, floats, half_step, inputs, product_limits, to_dev, weight
from f8_tiles import dw_form, dx_form, forward_tile
from gpu_util import say, torch_dev
from test_gpu_f8_backward import limits
from test_gpu_f8_gradient_range import behind_silu
from test_gpu_f8_linear import activated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


def operands(q8, m, n, k, parts):
    lib, torch, dev = q8
    rng = np.random.default_rng(m + n + k + parts)
    wq, wd, w = weight(rng, n, k, parts)
    xq, xd, x = inputs(rng, m, k)
    return rng, to_dev(torch, dev, wq, wd, xq, xd), w, x


# sizes, and the tile (weight rows, activation rows) of 16-bit and of float32 results
@pytest.mark.parametrize("m,n,k,narrow,wide", [
    (67, 8235, 944, (128, 64), (128, 64)), (260, 4117, 944, (128, 64), (128, 64)),
    (200, 8235, 944, (128, 128), (128, 128)), (515, 4117, 640, (128, 128), (128, 128)),
    (515, 7197, 944, (192, 256), (256, 128)), (1030, 4117, 640, (192, 256), (256, 128)),
    (1300, 8235, 944, (256, 256), (256, 128)), (1300, 8111, 640, (256, 256), (256, 128))])
def test_linear(q8, m, n, k, narrow, wide):
    lib, torch, dev = q8
    _, args, w, x = operands(q8, m, n, k, 1)
    for kind in TYPES:
        say(f"f8_linear m={m} n={n} k={k} {kind}")
        assert forward_tile(m, n, kind, False) == (wide if kind == "float32" else narrow)
        y = lib.f8_linear(*args, dtype=getattr(torch, kind))
        check(y, *product_limits(x, w, half_step(torch, kind)), f"f8_linear m={m} n={n} k={k} {kind}")


@pytest.mark.parametrize("m,f,k,narrow,wide", [
    (67, 4147, 944, (128, 64), (128, 64)), (150, 4147, 640, (128, 64), (128, 64)),
    (67, 8235, 944, (128, 128), (128, 128)), (260, 4117, 640, (128, 128), (128, 128)),
    (390, 8235, 944, (256, 256), (256, 128)), (515, 4117, 640, (256, 256), (256, 128))])
def test_gate_up(q8, m, f, k, narrow, wide):
    lib, torch, dev = q8
    _, args, w, x = operands(q8, m, f, k, 2)
    for kind in TYPES:
        say(f"f8 gate_up m={m} f={f} k={k} {kind}")
        assert forward_tile(m, f, kind, True) == (wide if kind == "float32" else narrow)
        half = half_step(torch, kind)
        h, gu = lib.f8_linear_fused_gate_up_silu(*args, dtype=getattr(torch, kind), keep_gate_up=True)
        check(gu, *product_limits(x, w, half), f"gate and up m={m} f={f} k={k} {kind}")
        check(h, *activated(*product_limits(x, w, 0.0, kind == "float32"), half), f"h m={m} f={f} k={k} {kind}")


# sizes, and how dx and dw run: large tiles, small ones, or small ones whose sums are cut into ranges
BACKWARD = [(150, 2100, 4112, "ranges", "large"), (700, 600, 4112, "small", "small"), (2100, 136, 4112, "large", "ranges")]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k,to_x,to_w", BACKWARD)
def test_linear_backward(q8, m, n, k, to_x, to_w, kind):
    lib, torch, dev = q8
    say(f"f8 backward m={m} n={n} k={k} {kind}")
    assert (dx_form(m, n, k, kind, 1), dw_form(m, n, k, kind, 1)) == (to_x, to_w)
    rng, args, w, x = operands(q8, m, n, k, 1)
    dy, d = as_type(torch, floats(rng, m, n), kind)
    dx, dw = lib.f8_linear_backward(*args, dy.to(dev))
    of_x, of_w = limits(d, w, x, kind, half_step(torch, kind))
    check(dx, *of_x, f"dx m={m} n={n} k={k} {kind}")
    check(dw, *of_w, f"dw m={m} n={n} k={k} {kind}")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,f,k,to_x,to_w", [(m, n // 2, k, to_x, to_w) for m, n, k, to_x, to_w in BACKWARD])
def test_gate_up_backward(q8, m, f, k, to_x, to_w, kind):
    lib, torch, dev = q8
    say(f"f8 gate_up backward m={m} f={f} k={k} {kind}")
    assert (dx_form(m, f, k, kind, 2), dw_form(m, f, k, kind, 2)) == (to_x, to_w)
    rng, args, w, x = operands(q8, m, f, k, 2)
    gu_t, gu = as_type(torch, 2 * floats(rng, m, 2 * f), kind)
    dh_t, dh = as_type(torch, floats(rng, m, f), kind)
    d, off = behind_silu(gu, dh, kind)
    dx, dw = lib.f8_linear_fused_gate_up_silu_backward(*args, gu_t.to(dev), dh_t.to(dev))
    of_x, of_w = limits(d, w, x, kind, half_step(torch, kind), off, off)
    check(dx, *of_x, f"dx m={m} f={f} k={k} {kind}")
    check(dw, *of_w, f"dw m={m} f={f} k={k} {kind}")
