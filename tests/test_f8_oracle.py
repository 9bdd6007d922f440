"""Pins of the 8-bit floating-point oracle: hand values of the code, rounding against brute force, the quantizer's rules."""

from __future__ import annotations

import numpy as np
import pytest

import oracle.f8_oracle as fo


def test_code_values():
    t = fo.e4m3_table()
    for code, value in {0x00: 0.0, 0x01: 2.0 ** -9, 0x07: 7 * 2.0 ** -9, 0x08: 2.0 ** -6, 0x38: 1.0, 0x39: 1.125,
                        0x40: 2.0, 0x7E: 448.0, 0x78: 256.0, 0xB8: -1.0, 0xFE: -448.0}.items():
        assert t[code] == value, hex(code)
    assert np.isnan(t[0x7F]) and np.isnan(t[0xFF]) and np.isfinite(np.delete(t, [0x7F, 0xFF])).all()
    torch = pytest.importorskip("torch")
    same = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(same, t, equal_nan=True)


def test_rounding_against_brute_force():
    rng = np.random.default_rng(1)
    t = fo.e4m3_table()[:127]
    mid = (t[1:] + t[:-1]) / 2
    v = np.concatenate([t, mid, mid * (1 + 2.0 ** -30), mid * (1 - 2.0 ** -30), rng.uniform(0, 448, 500),
                        2.0 ** rng.uniform(-12, 8, 500)])
    got = fo.e4m3_encode(v)
    for x, c in zip(v, got):
        off = np.abs(t - x)
        best = np.flatnonzero(off == off.min())
        assert c in best and (len(best) == 1 or c % 2 == 0), x
    assert np.array_equal(fo.e4m3_encode(-v), got | 128)


def test_quantizer_rules():
    x = np.zeros((3, 144), np.float32)
    x[0, :3] = [448.0, -1.0, 0.06]
    x[0, 130] = 7.0
    x[1, 0] = 2.0 ** -117
    x[2, 5], x[2, 143] = np.inf, 1.0
    q, d = fo.f8_quantize_ref(x, 1, False)
    assert d.shape == (3, 2) and d[0, 0] == 1.0 and d[0, 1] == np.float32(7.0) / np.float32(448.0)
    assert list(q[0, :4]) == [0x7E, 0xB8, fo.e4m3_encode(0.06), 0] and q[0, 130] == 0x7E
    assert d[1, 0] == 0 and not q[1].any()
    assert np.isnan(d[2, 0]) and (q[2, :128] == 0x7F).all() and np.isfinite(d[2, 1])
    for top, scale in ((448.0, 1.0), (448.1, 2.0), (224.0, 0.5), (1.0, 2.0 ** -8), (0.875, 2.0 ** -9)):
        assert fo.f8_quantize_ref(np.full((1, 16), top, np.float32), 1, True)[1][0, 0] == scale, top
    w = np.zeros((130, 130), np.float32)
    w[129, 0], w[0, 129] = 4.0, 2.0
    q, d = fo.f8_quantize_ref(w, 128, True)
    assert d.shape == (2, 2) and d[0, 0] == 0 and d[1, 0] == 2.0 ** -6 and d[0, 1] == 2.0 ** -7
    assert fo.f8_values(q, d, 128)[129, 0] == 4.0


def test_gradient_formula_against_differences():
    rng = np.random.default_rng(2)
    gu, dh = 2 * rng.standard_normal((4, 20)), rng.standard_normal((4, 10))
    d = fo.f8_gate_up_gradient_ref(gu, dh)
    step = 1e-6
    for c in range(20):
        e = np.zeros_like(gu)
        e[:, c] = step
        diff = ((fo.f8_gate_up_ref(gu + e) - fo.f8_gate_up_ref(gu - e)) * dh).sum(axis=1) / (2 * step)
        assert np.allclose(d[:, c], diff, rtol=1e-6, atol=1e-8)
