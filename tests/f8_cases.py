"""Inputs and error limits shared by the tests of the block-scaled 8-bit floating-point linears.

Limits, u = 2^-24.  A block's sum adds 128 exact products in float32; how the matrix cores round
inside is theirs, so each of its additions is counted with a whole step, 2u.  The block joins with
one rounding of the scales' product and one of the fma.  Worst case: (2 (127 + 1) + 2 + blocks) u
of the sum of the terms' magnitudes.  In the norm the roundings have random signs and are a part of
a partial sum no larger than the root of the terms' squares (in the mean): u sqrt(4 * 128 + 2 +
blocks) of that root.  A result's own rounding is at most finfo(type).eps / 2 of it."""

from __future__ import annotations

import numpy as np

import oracle.f8_oracle as fo

U = 2.0 ** -24
TYPES = ["float32", "float16", "bfloat16"]


def half_step(torch, kind):
    return torch.finfo(getattr(torch, kind)).eps / 2


def floats(rng, *shape):
    return rng.standard_normal(shape).astype(np.float32)


def as_type(torch, x, kind):
    """(tensor of the type on the CPU, its values in float64)"""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(getattr(torch, kind))
    return t, t.to(torch.float64).numpy()


def weight(rng, n, k, parts=1, pow2=False):
    """(codes, scales, values) of a matrix of `parts` parts of n rows each, of about N(0, 0.05^2)."""
    coded = [fo.f8_quantize_ref(0.05 * floats(rng, n, k), fo.F8_BLOCK, pow2) for _ in range(parts)]
    q, d = np.concatenate([c[0] for c in coded]), np.concatenate([c[1] for c in coded])
    return q, d, fo.f8_weight_values(q, d, parts)


def inputs(rng, m, k, pow2=False):
    q, d = fo.f8_quantize_ref(floats(rng, m, k), 1, pow2)
    return q, d, fo.f8_values(q, d, 1)


def to_dev(torch, dev, *arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).to(dev) for a in arrays]


def rounding(half, size):
    """What a result of magnitude `size` may be off by its type's rounding: half a step, which for a
    binary16 result (half = 2^-11) below 2^-14 is the half of 2^-24, the step of its subnormals."""
    return np.maximum(half * size, 2.0 ** -25 if half == 2.0 ** -11 else 0.0)


def product_limits(x, w, half, wide=None):
    """(x . w^T, the largest error of each output, the expected size of it) in float64; half: the
    results' rounding, wide: whether the sums are of float32 accuracy (a float32 result's)."""
    wide = half <= U if wide is None else wide
    y = x @ w.T
    blocks = -(-x.shape[1] // 128)
    worst = U * (2 * 128 + 2 + blocks) * (np.abs(x) @ np.abs(w).T)
    usual = U * np.sqrt(4 * 128 + 2 + blocks) * np.sqrt(x ** 2 @ (w ** 2).T)
    if not wide:
        worst = worst + 2.0 ** -10 * (np.abs(x) @ np.abs(w).T)
        usual = usual + 2.0 ** -13 * np.sqrt(x ** 2 @ (w ** 2).T)
    return y, worst + rounding(half, np.abs(y) + worst), usual + rounding(half, np.abs(y))


def check(got, want, worst, usual, what):
    """Every element within its largest error, and the error's norm within the usual ones'."""
    got = got.double().cpu().numpy() if hasattr(got, "cpu") else np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), what
    off = np.abs(got - want)
    part = np.linalg.norm(off) / max(np.linalg.norm(usual), 1e-300)
    print(f"[gpu-test] {what}: worst {np.max(off / np.maximum(worst, 1e-300), initial=0):.3f} of its limit, "
          f"norm {part:.3f}", flush=True)
    assert (off <= worst).all(), (what, np.max(off - worst))
    assert part <= 1, (what, part)
