"""The adapter calls are of float32 accuracy in the norm, not within worst-case bounds alone.

A worst-case bound (test_gpu_lora.py) adds up every rounding with one sign and the terms'
magnitudes: at long rows it would let whole parts of the operands go missing.  Here the
error's norm is held against the size that sums of these (random) terms really have.

With u = 2^-24, a sum whose terms pass through at most d roundings of random sign, each at
most u of a partial sum that is no larger than the root of its terms' squares, is off by at
most u sqrt(d) of that root in the mean square; sqrt(d) also covers the tail, the mean square
of a rounding being a third of its largest.  Beside that stand parts with one sign, at their
largest: the products left out where a factor is taken as three bf16 parts, 2^-21 = 8 u for
each of the two products of an adapter (16 u); for the shared product 8 u, the fixed-point rounding of
x (2^-30 of the row's largest, u / 64, times the square root of the terms where one weight
meets it) and a sum's and a scale's last roundings.  d: as in test_gpu_lora.py."""

from __future__ import annotations

import numpy as np
import pytest
import torch as torch_cpu

import oracle
import workloads as wl
from gpu_util import say, to_dev, torch_dev
from test_gpu_lora import LINEARS, MANY, TYPES, Case, packed

U = 2.0 ** -24


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


def delta(c, cut=lambda v: v):
    """(D, the size of its sums), [m][n] float64; cut: what is done to every factor."""
    d, size = np.zeros((c.m, c.n)), np.zeros((c.m, c.n))
    x = cut(c.x.astype(np.float64))
    for t, e in enumerate(c.adapter):
        if not 0 <= e < c.count:
            continue
        r = c.rank if c.ranks is None else int(c.ranks[e])
        at = 0
        for p, rows in enumerate(c.parts):
            a, b = c.a64[e, p * c.rank:p * c.rank + r], c.b64[e, at:at + rows, :r]
            u = c.scale[e].astype(np.float64) * (cut(a) @ x[t])
            d[t, at:at + rows] = cut(b) @ cut(u)
            size[t, at:at + rows] = abs(c.scale[e]) * np.sqrt(b ** 2 @ (a ** 2 @ c.x[t].astype(np.float64) ** 2))
            at += rows
    return d, size


def delta_tol(c):
    return U * (np.sqrt(c.k / 8 + 16 + c.rank + 4) + 16)


def product(w64, x):
    x = x.astype(np.float64)
    return x @ w64.T, np.sqrt(x ** 2 @ (w64 ** 2).T)


def product_tol(k):
    return U * (np.sqrt(k / 32 + 52) + 8)


def within(got, want, off_at_most, what):
    """The norm of the error against that of the elements' expected errors; nothing else."""
    off = np.linalg.norm(np.asarray(got, np.float64) - want)
    most = np.linalg.norm(off_at_most)
    say(f"{what}: error {off / max(np.linalg.norm(want), 1e-300):.1e} of the norm, {off / max(most, 1e-300):.3f} of its limit")
    return off <= most


def activated(v, ve, f):
    """As in test_gpu_lora.py: |SiLU'| <= 1.1, the activation's own (|g| + 8) 2^-23."""
    g, u, ge, ue = v[:, :f], v[:, f:], ve[:, :f], ve[:, f:]
    s = oracle.silu_ref(g)
    return s * u, 1.1 * np.abs(u) * ge + np.abs(s) * ue + (np.abs(g) + 8) * 2.0 ** -23 * np.abs(s * u)


def expected(c, w64):
    """(y + D, the elements' expected errors)"""
    y, ys = product(w64, c.x)
    d, ds = delta(c)
    return y + d, product_tol(c.k) * ys + delta_tol(c) * ds + U * np.abs(y + d)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n,k,count,rank,sections", LINEARS)
def test_linear(q8, m, n, k, count, rank, sections):
    lib, torch, dev = q8
    c = Case(q8, 6000 + m + n, m, n, k, count, rank, TYPES[(m + n + 1) % 3], sections)
    w, w64 = packed(6001 + n, n, k)
    y = lib.q8_linear_lora(to_dev(w, dev), n, k, c.xd, *c.args, **c.more)
    assert within(y.cpu(), *expected(c, w64), f"q8_linear_lora m={m} n={n} k={k}")


@pytest.mark.gpu
@pytest.mark.parametrize("m,f,k,count,rank,split", [(1, 128, 1024, 1, 16, True), (3, 90, 12288, 2, 64, True),
                                                    (8, 500, 2048, 4, 32, True), (21, 40, 4096, 3, 8, False),
                                                    (255, 33, 512, 9, 24, True), (4, 19, 16640, 2, 8, True)])
def test_gate_up(q8, m, f, k, count, rank, split):
    lib, torch, dev = q8
    c = Case(q8, 6100 + m + f, m, 2 * f, k, count, rank, TYPES[(m + f) % 3], [f, f] if split else None)
    # gate and up of the size of activations, or every SiLU would be at one of its ends
    c.x = (c.x / np.float32(64 * np.sqrt(k) / 16)).astype(np.float32)
    c.xd = to_dev(c.x, dev)
    w, w64 = packed(6101 + f, 2 * f, k)
    h = lib.q8_linear_fused_gate_up_silu_lora(to_dev(w, dev), f, k, c.xd, *c.args, **c.more)
    assert within(h.cpu(), *activated(*expected(c, w64), f), f"gate_up m={m} f={f} k={k}")


FEW = [(1, 300, 256, 2, 8, None), (7, 65, 512, 3, 16, [1, 64]), (40, 200, 16384, 2, 24, [72, 128]),
       (130, 515, 2048, 3, 64, [256, 259]), (300, 64, 512, 4, 256, None)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k,count,rank,sections", FEW + MANY)
def test_add(q8, m, n, k, count, rank, sections, kind):
    """Beside a product of zeros: the correction alone."""
    lib, torch, dev = q8
    c = Case(q8, 6200 + m + n, m, n, k, count, rank, kind, sections)
    out = lib.lora_add(torch.zeros((m, n), device=dev), c.xd, *c.args, **c.more)
    d, size = delta(c)
    assert within(out.cpu(), d, delta_tol(c) * size, f"lora_add m={m} n={n} k={k} rank={rank} {kind}")


@pytest.mark.gpu
@pytest.mark.parametrize("m,f,k,count,rank", [(6, 33, 512, 3, 16), (420, 77, 1280, 7, 96), (1100, 301, 512, 30, 64),
                                              (48, 65, 8192, 2, 256)])
@pytest.mark.parametrize("kind", TYPES)
def test_act(q8, m, f, k, count, rank, kind):
    lib, torch, dev = q8
    c = Case(q8, 6300 + m + f, m, 2 * f, k, count, rank, kind, [f, f])
    gu = wl.activations(6301 + m, m, 2 * f)
    h = lib.lora_gate_up_silu(to_dev(gu, dev), c.xd, *c.args, **c.more)
    d, size = delta(c)
    v = gu.astype(np.float64) + d
    assert within(h.cpu(), *activated(v, delta_tol(c) * size + U * np.abs(v), f), f"lora_gate_up_silu m={m} f={f} {kind}")


# ---------------------------------------------- the limits see what they are for (CPU)


def cut_parts(parts):
    """v cut to its first `parts` bf16 parts of eight bits."""
    def cut(v):
        bits = np.ascontiguousarray(v, dtype=np.float32).view(np.uint32)
        whole = np.zeros(v.shape)
        rest = bits.view(np.float32)
        for _ in range(parts):
            lead = (np.ascontiguousarray(rest).view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
            whole += lead
            rest = (rest - lead).astype(np.float32)
        return whole
    return cut


@pytest.mark.parametrize("m,n,k,count,rank,sections", [s for s in MANY if s[0] <= 1300])
def test_limits_see_a_part_too_few(m, n, k, count, rank, sections):
    c = Case((None, torch_cpu, torch_cpu.device("cpu")), 6200 + m + n, m, n, k, count, rank, "float32", sections)
    d, size = delta(c)
    assert within(delta(c, cut_parts(3))[0], d, delta_tol(c) * size, "three parts")
    assert not within(delta(c, cut_parts(2))[0], d, delta_tol(c) * size, "two parts")


@pytest.mark.parametrize("n,k", [(64, 1024), (40, 8192), (24, 16384)])
def test_limits_see_digits_that_are_missing(n, k):
    x = wl.activations(6400, 5, k).astype(np.float64)
    _, w64 = packed(6401, n, k)
    y, size = product(w64, x)
    top = 2.0 ** np.floor(np.log2(np.abs(x).max(axis=1, keepdims=True)))
    for digits, fine in ((4, True), (2, False)):
        step = top * 2.0 ** (-29 + 8 * (4 - digits))
        assert within((np.round(x / step) * step) @ w64.T, y, product_tol(k) * size, f"{digits} digits") == fine
