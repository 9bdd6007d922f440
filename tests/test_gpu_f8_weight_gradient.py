"""dw takes x's values (code * scale) to 2^-16 and better with gradients of every type: what a 16-bit dw is off by is its
own rounding, and behind the activation that of dg and du where they are of bf16.

A rounding to nearest is uniform within a step: 1/sqrt(12) of it in the mean.  Roundings of N independent numbers have a
norm within 4 / sqrt(N) of their mean's (the variance of a square is 4/5 of the square of its mean).  The sums' own part is
`usual` of test_gpu_f8_backward.py, with x off by 2^-16."""

from __future__ import annotations

import numpy as np
import pytest

from f8_cases import U, as_type, floats, half_step, inputs, to_dev, weight
from gpu_util import say, torch_dev
from test_gpu_f8_backward import LEFT_OUT, TERMS
from test_gpu_f8_gradient_range import D_OFF, behind_silu

pytestmark = pytest.mark.gpu

SHAPES = [(63, 130, 256), (130, 48, 2064), (300, 2100, 4112), (700, 600, 4112)]


def step(v, half):
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -100)))) * 2 * half


def expected(d, x, kind, half, d_off=0.0):
    """(dw, the norm that its error may have); d_off: what d's elements are off by in the mean"""
    m, n = d.shape
    want = d.T @ x
    own = np.linalg.norm(step(want, half)) / np.sqrt(12) * (1 + 4 / np.sqrt(want.size))
    before = np.sqrt((np.broadcast_to(d_off, d.shape) ** 2).T @ x ** 2)
    before = np.linalg.norm(before) * (1 + 4 / np.sqrt(d.size))
    adds = 2 * TERMS[kind] * (TERMS[kind] + 1) // 2 * (m + 64) * 2
    sums = np.sqrt(2 * U * U * adds + (2.0 ** -16 + LEFT_OUT[kind]) ** 2) * np.linalg.norm(np.sqrt((d ** 2).T @ x ** 2))
    return want, np.sqrt(own ** 2 + before ** 2 + sums ** 2)


def check(dw, want, allowed, what):
    off = np.linalg.norm(dw.double().cpu().numpy() - want)
    say(f"{what}: off by {off / np.linalg.norm(want):.3e} of the norm, {allowed / np.linalg.norm(want):.3e} allowed")
    assert off <= allowed


@pytest.mark.parametrize("kind", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(m, n, k, kind):
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8
    rng = np.random.default_rng(m + n + k + 3)
    (wq, wd, _), (xq, xd, x) = weight(rng, n, k), inputs(rng, m, k)
    dy, d = as_type(torch, floats(rng, m, n), kind)
    _, dw = q8.f8_linear_backward(*to_dev(torch, dev, wq, wd, xq, xd), dy.to(dev), dx=False)
    check(dw, *expected(d, x, kind, half_step(torch, kind)), f"dw m={m} n={n} k={k} {kind}")


@pytest.mark.parametrize("kind", ["bfloat16", "float16"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gate_up(m, n, k, kind):
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8
    rng = np.random.default_rng(m + n + k + 4)
    f = n // 2
    (wq, wd, _), (xq, xd, x) = weight(rng, f, k, parts=2), inputs(rng, m, k)
    gu_t, gu = as_type(torch, 2 * floats(rng, m, 2 * f), kind)
    dh_t, dh = as_type(torch, floats(rng, m, f), kind)
    d, off = behind_silu(gu, dh, kind)
    off = off - D_OFF[kind] * np.abs(d) + (step(d, 2.0 ** -8) / np.sqrt(12) if kind == "bfloat16" else D_OFF[kind] * np.abs(d))
    _, dw = q8.f8_linear_fused_gate_up_silu_backward(*to_dev(torch, dev, wq, wd, xq, xd), gu_t.to(dev), dh_t.to(dev), dx=False)
    check(dw, *expected(d, x, kind, half_step(torch, kind), off), f"dw m={m} f={f} k={k} {kind}")
