"""Gradients behind SiLU(gate) * up whose values between the activation and the products pass the range of the
call's type, in either direction, where the results lie within it.

Limits as in test_gpu_f8_backward.py.  The activation's gradients are held in float32 (its own roundings: (|g| + 10) 2u of
their parts) and enter the products as 1, 2 or 3 bf16 parts, each to nearest: off by 2^-8 with bf16 gradients, 2^-17
with binary16 ones (half a step of eight bits, twice, is 2^-18), and not at all with float32 ones."""

from __future__ import annotations

import numpy as np
import pytest

import oracle.f8_oracle as fo
from f8_cases import TYPES, U, as_type, check, floats, half_step, inputs, to_dev, weight
from gpu_util import say, torch_dev
from test_gpu_f8_backward import limits

pytestmark = pytest.mark.gpu

D_OFF = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -17, "float32": 0.0}


def behind_silu(gu, dh, kind):
    """([dg du], what its elements are off by where they enter the products) in float64."""
    f = dh.shape[1]
    g, u = np.abs(gu[:, :f]), np.abs(gu[:, f:])
    s = 1 / (1 + np.exp(-gu[:, :f]))
    parts = np.concatenate([np.abs(dh) * u * s * (1 + g * (1 - s)), np.abs(dh) * g * s], axis=1)
    own = 2 * U * (np.concatenate([g, g], axis=1) + 10) * parts
    d = fo.f8_gate_up_gradient_ref(gu, dh)
    return d, D_OFF[kind] * (np.abs(d) + own) + own


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,f,k", [(1, 20, 144), (70, 129, 272), (300, 2100, 4112)])
@pytest.mark.parametrize("size,w_by,x_by", [(2e4, 2.0 ** -9, 2.0 ** -9), (1e-6, 2.0 ** 8, 2.0 ** 8)])
def test_gate_up(size, w_by, x_by, m, f, k, kind):
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8
    say(f"f8 gate_up backward, gradients of {size}, m={m} f={f} k={k} {kind}")
    rng = np.random.default_rng(m + f + k + 2)
    wq, wd, w = weight(rng, f, k, parts=2)
    xq, xd, x = inputs(rng, m, k)
    wd, w, xd, x = wd * np.float32(w_by), w * w_by, xd * np.float32(x_by), x * x_by
    gu_t, gu = as_type(torch, 2 * floats(rng, m, 2 * f), kind)
    dh_t, dh = as_type(torch, np.float32(size) * np.clip(floats(rng, m, f), -3, 3), kind)
    half = half_step(torch, kind)
    d, off = behind_silu(gu, dh, kind)
    if m > 1:  # the point of the test: binary16 does not hold d
        assert np.abs(d).max() > 65504 if size > 1 else np.median(np.abs(d)) < 2.0 ** -20
    dx, dw = q8.f8_linear_fused_gate_up_silu_backward(*to_dev(torch, dev, wq, wd, xq, xd), gu_t.to(dev), dh_t.to(dev))
    to_x, to_w = limits(d, w, x, kind, half, off, off)
    assert max(np.abs(to_x[0]).max(), np.abs(to_w[0]).max()) < 6e4
    check(dx, *to_x, f"dx m={m} f={f} k={k} {kind}")
    check(dw, *to_w, f"dw m={m} f={f} k={k} {kind}")
