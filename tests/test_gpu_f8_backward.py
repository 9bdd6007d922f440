"""The gradients of the 8-bit floating-point linears against the float64 oracle and differences.

Limits, u = 2^-24 (f8_cases.py): a product of parts is exact; dx adds 64 of them from zero (2u each),
joins with the scale's fma (u), over parts * terms * ceil(n/64) steps; dw adds all of its products to
one sum (2u each).  Operands: bf16 gradients 1 part, binary16 2, float32 3; a value of x is off by
2^-8 (the half step of bf16), 2^-17, 0 of itself, and products of parts of 0, 2^-16, 2^-24 are left
out.  A gradient behind the activation is off by its own rounding and by (|g| + 10) 2u."""

from __future__ import annotations

import numpy as np
import pytest

import oracle.f8_oracle as fo
from f8_cases import TYPES, U, as_type, check, floats, half_step, inputs, rounding, to_dev, weight
from gpu_util import say, torch_dev

pytestmark = pytest.mark.gpu

TERMS = {"bfloat16": 1, "float16": 2, "float32": 3}
X_OFF = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -17, "float32": 0.0}
LEFT_OUT = {"bfloat16": 0.0, "float16": 2.0 ** -16, "float32": 2.0 ** -24}


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


def limits(d, w, x, kind, half, d_worst=None, d_usual=None, pow2=False):
    """((dx, worst, usual), (dw, worst, usual)); d_*: what d's elements are off by already."""
    m, n = d.shape
    terms = TERMS[kind]
    d_worst = np.zeros_like(d) if d_worst is None else d_worst
    d_usual = np.zeros_like(d) if d_usual is None else d_usual
    a, out = np.abs, []
    steps = terms * (n // 64 + 2)
    x_off = 0.0 if pow2 else X_OFF[kind]
    for d1, o, count, off, left in ((d, w, 2 * 64 + steps + 2, 0.0, 0.0),
                                    (d.T, x, 2 * terms * (terms + 1) // 2 * (m + 64), x_off, LEFT_OUT[kind])):
        dw1, du1 = (d_worst, d_usual) if d1 is d else (d_worst.T, d_usual.T)
        y = d1 @ o
        worst = (1.02 * U * count + off + left) * (a(d1) @ a(o)) + 1.01 * (dw1 @ a(o))
        usual = np.sqrt((2 * U * U * count + (off + left) ** 2) * (d1 ** 2 @ o ** 2) + du1 ** 2 @ o ** 2)
        out.append((y, worst + rounding(half, a(y) + worst), usual + rounding(half, a(y))))
    return out


SHAPES = [(1, 1, 16), (1, 300, 1040), (2, 64, 128), (7, 130, 272), (63, 129, 256), (64, 257, 144), (65, 1000, 384),
          (130, 48, 2064), (200, 515, 640), (321, 264, 1296), (700, 1300, 400)]
# from here on the calls take the large tiles
LARGE = [(2100, 300, 4112, "bfloat16"), (1290, 136, 6416, "float16"), (300, 2100, 4112, "bfloat16")]
CASES = [(*s, kind) for s in SHAPES for kind in TYPES] + LARGE


@pytest.mark.parametrize("m,n,k,kind", CASES)
def test_linear(q8, m, n, k, kind):
    lib, torch, dev = q8
    say(f"f8 backward m={m} n={n} k={k} {kind}")
    rng = np.random.default_rng(m + n + k)
    wq, wd, w = weight(rng, n, k)
    xq, xd, x = inputs(rng, m, k)
    dy, d = as_type(torch, floats(rng, m, n), kind)
    args = to_dev(torch, dev, wq, wd, xq, xd)
    dx, dw = lib.f8_linear_backward(*args, dy.to(dev))
    to_x, to_w = limits(d, w, x, kind, half_step(torch, kind))
    check(dx, *to_x, f"dx m={m} n={n} k={k} {kind}")
    check(dw, *to_w, f"dw m={m} n={n} k={k} {kind}")


@pytest.mark.parametrize("m,f,k,kind", CASES)
def test_gate_up(q8, m, f, k, kind):
    lib, torch, dev = q8
    say(f"f8 gate_up backward m={m} f={f} k={k} {kind}")
    rng = np.random.default_rng(m + f + k + 1)
    wq, wd, w = weight(rng, f, k, parts=2)
    xq, xd, x = inputs(rng, m, k)
    gu_t, gu = as_type(torch, 2 * floats(rng, m, 2 * f), kind)
    dh_t, dh = as_type(torch, floats(rng, m, f), kind)
    half = half_step(torch, kind)
    d = fo.f8_gate_up_gradient_ref(gu, dh)
    g, u = np.abs(gu[:, :f]), np.abs(gu[:, f:])
    # the activation's roundings are relative to the parts of dg: s (1 + |g| (1 - s)), not to what is left of them
    s = 1 / (1 + np.exp(-gu[:, :f]))
    parts = np.concatenate([np.abs(dh) * u * s * (1 + g * (1 - s)), np.abs(dh) * g * s], axis=1)
    own = 2 * U * (np.concatenate([g, g], axis=1) + 10) * parts
    off = rounding(half, np.abs(d) + own) + own
    dx, dw = lib.f8_linear_fused_gate_up_silu_backward(*to_dev(torch, dev, wq, wd, xq, xd), gu_t.to(dev), dh_t.to(dev))
    to_x, to_w = limits(d, w, x, kind, half, off, off)
    check(dx, *to_x, f"dx m={m} f={f} k={k} {kind}")
    check(dw, *to_w, f"dw m={m} f={f} k={k} {kind}")


@pytest.mark.parametrize("m,n,k", [(1, 130, 272), (64, 128, 256), (100, 300, 400), (700, 333, 4112), (2100, 72, 4112)])
@pytest.mark.parametrize("kind", TYPES)
def test_exact_sums(q8, m, n, k, kind):
    """Small whole numbers and scales that are powers of two: exact in every part and sum."""
    lib, torch, dev = q8
    say(f"exact backward m={m} n={n} k={k} {kind}")
    rng = np.random.default_rng(m + n)
    kb, nb = -(-k // 128), -(-n // 128)
    wq, xq = fo.e4m3_encode(rng.integers(-3, 4, (n, k))), fo.e4m3_encode(rng.integers(-1, 2, (m, k)))
    wd, xd = 2.0 ** rng.integers(0, 2, (nb, kb)), 2.0 ** rng.integers(0, 2, (m, kb))
    # few gradients are not zero, so that sums stay within the type
    dy = rng.integers(-1, 2, (m, n)) * (rng.random((m, n)) < 0.02)
    w, x = fo.f8_values(wq, wd, 128), fo.f8_values(xq, xd, 1)
    args = to_dev(torch, dev, wq, wd.astype(np.float32), xq, xd.astype(np.float32))
    dx, dw = lib.f8_linear_backward(*args, torch.from_numpy(dy).to(dev, getattr(torch, kind)))
    assert max(np.abs(dy @ w).max(), np.abs(dy.T @ x).max()) <= 256
    assert np.array_equal(dx.double().cpu().numpy(), dy @ w)
    assert np.array_equal(dw.double().cpu().numpy(), dy.T @ x)


def test_differences(q8):
    """The gradient of sum(h * dh) from the forward call at x and at x +- step, in float32."""
    lib, torch, dev = q8
    rng = np.random.default_rng(3)
    m, f, k = 3, 40, 128
    wq, wd, w = weight(rng, f, k, parts=2, pow2=True)
    xq, xd, x = inputs(rng, m, k, pow2=True)
    dh = rng.standard_normal((m, f))
    args = to_dev(torch, dev, wq, wd, xq, xd)
    _, gu = lib.f8_linear_fused_gate_up_silu(*args, keep_gate_up=True)
    dx, _ = lib.f8_linear_fused_gate_up_silu_backward(*args, gu, torch.from_numpy(dh).to(dev, torch.float32))
    step = 2.0 ** -10
    for i in rng.choice(k, 12, replace=False):
        moved = [fo.f8_gate_up_ref((x + s * np.eye(k)[i]) @ w.T) for s in (step, -step)]
        diff = ((moved[0] - moved[1]) * dh).sum(axis=1) / (2 * step)
        # the third derivative's share is step^2 of numbers of order one; float32's own is below 1e-5
        assert np.allclose(dx[:, i].cpu().numpy(), diff, rtol=1e-4, atol=1e-4)


def test_parts_of_the_call(q8):
    """One gradient alone has the bits that both together have; strided operands and outputs; a caller's workspace."""
    lib, torch, dev = q8
    rng = np.random.default_rng(4)
    for m, n, k in ((5, 37, 272), (130, 256, 384)):
        wq, wd, xq, xd = to_dev(torch, dev, *weight(rng, n, k)[:2], *inputs(rng, m, k)[:2])
        for kind in TYPES:
            dtype = getattr(torch, kind)
            dy = torch.randn(m, n, device=dev).to(dtype)
            dx, dw = lib.f8_linear_backward(wq, wd, xq, xd, dy)
            assert torch.equal(lib.f8_linear_backward(wq, wd, xq, xd, dy, dw=False)[0], dx)
            assert torch.equal(lib.f8_linear_backward(wq, wd, xq, xd, dy, dx=False)[1], dw)
            assert lib.f8_linear_backward(wq, wd, xq, xd, dy, dx=False, dw=False) == (None, None)
            wide = torch.full((m * (n + 3) + 1,), float("nan"), dtype=dtype, device=dev)
            view = wide[1:].view(m, n + 3)[:, :n]
            view.copy_(dy)
            ox = torch.full((m, k + 1), -7.0, dtype=dtype, device=dev)
            ow = torch.full((n, k + 5), -7.0, dtype=dtype, device=dev)
            need = lib.f8_linear_backward_workspace_bytes(m, n, k, dtype)
            ws = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=dev)
            lib.f8_linear_backward(wq, wd, xq, xd, view, dx=ox[:, :k], dw=ow[:, :k], workspace=ws[:need])
            assert torch.equal(ox[:, :k], dx) and (ox[:, k:] == -7).all()
            assert torch.equal(ow[:, :k], dw) and (ow[:, k:] == -7).all()
            assert (ws[need:] == 0xFF).all()


def test_empty_sums_are_zeros(q8):
    lib, torch, dev = q8
    rng = np.random.default_rng(5)
    wq, wd, xq, xd = to_dev(torch, dev, *weight(rng, 20, 160, parts=2)[:2], *inputs(rng, 4, 160)[:2])
    ow = torch.full((40, 168), -7.0, device=dev)
    dx, dw = lib.f8_linear_fused_gate_up_silu_backward(wq, wd, xq[:0], xd[:0], torch.empty(0, 40, device=dev),
                                                       torch.empty(0, 20, device=dev), dw=ow[:, :160])
    assert dx.shape == (0, 160) and (dw == 0).all() and (ow[:, 160:] == -7).all()
    dx, dw = lib.f8_linear_backward(wq[:0], wd[:0], xq, xd, torch.empty(4, 0, device=dev))
    assert dw.shape == (0, 160) and dx.shape == (4, 160) and (dx == 0).all()


@pytest.mark.parametrize("kind", TYPES)
def test_not_finite_stays_in_its_place(q8, kind):
    lib, torch, dev = q8
    rng = np.random.default_rng(6)
    m, n, k = 70, 129, 272
    wq, wd, xq, xd = to_dev(torch, dev, *weight(rng, n, k)[:2], *inputs(rng, m, k)[:2])
    dy = torch.randn(m, n, device=dev).to(getattr(torch, kind))
    dx, dw = lib.f8_linear_backward(wq, wd, xq, xd, dy)
    for value in ("nan", "inf"):
        bad = dy.clone()
        bad[69, 128] = float(value)  # the last row and column
        bx, bw = lib.f8_linear_backward(wq, wd, xq, xd, bad)
        assert not torch.isfinite(bx[69]).any() and torch.equal(bx[:69], dx[:69])
        assert not torch.isfinite(bw[128]).any() and torch.equal(bw[:128], dw[:128])
    codes = wq.clone()
    codes[128, 271] = 0x7F
    bx, bw = lib.f8_linear_backward(codes, wd, xq, xd, dy)
    assert torch.isnan(bx[:, 271]).all() and torch.equal(bx[:, :271], dx[:, :271]) and torch.equal(bw, dw)
    codes = xq.clone()
    codes[69, 0] = 0xFF
    bx, bw = lib.f8_linear_backward(wq, wd, codes, xd, dy)
    assert torch.isnan(bw[:, 0]).all() and torch.equal(bw[:, 1:], dw[:, 1:]) and torch.equal(bx, dx)


def test_large_and_small_gradients(q8):
    """Float32 gradients at the ends of their range keep their parts."""
    lib, torch, dev = q8
    rng = np.random.default_rng(7)
    wq, wd, xq, xd = to_dev(torch, dev, fo.e4m3_encode(np.eye(32)), np.ones((1, 1), np.float32),
                            fo.e4m3_encode(np.ones((1, 32))), np.ones((1, 1), np.float32))
    dy = np.concatenate([[3.4028235e38, -3.4e38], 2.0 ** rng.uniform(-100, 127, 30)]).astype(np.float32)[None]
    dx, dw = lib.f8_linear_backward(wq, wd, xq, xd, torch.from_numpy(dy).to(dev))
    assert np.array_equal(dx.cpu().numpy(), dy)
    assert np.array_equal(dw.cpu().numpy(), dy.T.repeat(32, axis=1))


def test_refusals(q8):
    lib, torch, dev = q8
    rng = np.random.default_rng(8)
    wq, wd, xq, xd = to_dev(torch, dev, *weight(rng, 20, 160, parts=2)[:2], *inputs(rng, 4, 160)[:2])
    back, gate = lib.f8_linear_backward, lib.f8_linear_fused_gate_up_silu_backward
    dy, dh, gu = (torch.zeros(4, c, device=dev) for c in (40, 20, 40))
    one = wd[:1]
    for bad in (torch.zeros(4, 39, device=dev), torch.zeros(3, 40, device=dev), dy.double(), dy.cpu(), dy.t()):
        with pytest.raises(ValueError):
            back(wq, one, xq, xd, bad)
    for bad in ((gu[:, :39], dh), (gu.half(), dh), (gu, dh[:, :19]), (gu[:3], dh), (gu.cpu(), dh)):
        with pytest.raises(ValueError):
            gate(wq, wd, xq, xd, *bad)
    with pytest.raises(ValueError):
        back(wq, one, xq, xd, dy, dx=torch.empty(4, 161, device=dev))
    with pytest.raises(ValueError):
        back(wq, one, xq, xd, dy, dw=torch.empty(40, 160, device=dev, dtype=torch.float16))
    with pytest.raises(lib.Q8Error):
        back(wq, one, xq, xd, dy, workspace=torch.empty(256, dtype=torch.uint8, device=dev))


def test_repeats_streams_and_graphs(q8):
    lib, torch, dev = q8
    rng = np.random.default_rng(9)
    for m, f, k in ((1, 100, 272), (90, 136, 528), (1100, 264, 4112)):
        wq, wd, xq, xd = to_dev(torch, dev, *weight(rng, f, k, parts=2)[:2], *inputs(rng, m, k)[:2])
        gu, dh = torch.randn(m, 2 * f, device=dev).bfloat16(), torch.randn(m, f, device=dev).bfloat16()
        want = lib.f8_linear_fused_gate_up_silu_backward(wq, wd, xq, xd, gu, dh)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = lib.f8_linear_fused_gate_up_silu_backward(wq, wd, xq, xd, gu, dh)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(other, want))
        dx, dw = (torch.empty_like(t) for t in want)
        ws = torch.empty(lib.f8_linear_fused_gate_up_silu_backward_workspace_bytes(m, f, k, torch.bfloat16),
                         dtype=torch.uint8, device=dev)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.f8_linear_fused_gate_up_silu_backward(wq, wd, xq, xd, gu, dh, dx=dx, dw=dw, workspace=ws)
        for turn in range(4):
            gu.copy_(torch.randn(m, 2 * f, device=dev))
            dh.copy_(torch.randn(m, f, device=dev))
            ws.fill_(0xFF)
            graph.replay()
            torch.cuda.synchronize()
            eager = lib.f8_linear_fused_gate_up_silu_backward(wq, wd, xq, xd, gu, dh)
            assert torch.equal(dx, eager[0]) and torch.equal(dw, eager[1]), turn
