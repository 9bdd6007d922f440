"""The 8-bit floating-point quantizers, linear and fused gate_up against the float64 oracle."""

from __future__ import annotations

import numpy as np
import pytest

import oracle.f8_oracle as fo
from f8_cases import TYPES, U, as_type, check, floats, half_step, inputs, product_limits, rounding, to_dev, weight
from gpu_util import say, torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


# ------------------------------------------------------------------------- quantizers


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,k", [(1, 16), (3, 144), (17, 1040), (130, 256), (257, 4096)])
def test_quantize(q8, m, k, kind, pow2):
    """Bit for bit, blocks of both shapes, a strided operand, ties and tiny blocks among the values."""
    lib, torch, dev = q8
    say(f"quantize m={m} k={k} {kind} pow2={pow2}")
    rng = np.random.default_rng(m + k)
    x = floats(rng, m, k) * np.float32(2.0) ** rng.integers(-12, 12, (m, 1)).astype(np.float32)
    x[0, : k // 2] = rng.integers(-448, 449, k // 2) / 2  # many of these fall between two codes
    x[0, 0] = 448.0
    x[m // 2, :16] = 0
    if m > 2:
        x[2] *= np.float32(2.0 ** -20)
    t, v = as_type(torch, x, kind)
    wide = torch.full((m, k + 24), 7e4 if kind == "float16" else 1e30).to(t.dtype)
    wide[:, :k] = t
    xd = wide.to(dev)[:, :k]
    for fn, rows in ((lib.f8_quantize_act, 1), (lib.f8_quantize_weight, 128)):
        q, d = fn(xd, pow2=pow2)
        rq, rd = fo.f8_quantize_ref(v, rows, pow2)
        assert q.dtype == torch.float8_e4m3fn and np.array_equal(d.cpu().numpy(), rd)
        assert np.array_equal(q.view(torch.uint8).cpu().numpy(), rq)


def test_quantize_special_values(q8):
    lib, torch, dev = q8
    x = np.ones((6, 272), np.float32)
    x[0] = 0
    x[1, 3] = np.nan
    x[2, 200] = -np.inf
    x[3] = np.float32(2.0 ** -117)
    x[4] = np.float32(3.4e38)
    x[5, 128:256] = np.float32(2.0 ** -116)
    for pow2 in (False, True):
        for fn, rows in ((lib.f8_quantize_act, 1), (lib.f8_quantize_weight, 128)):
            q, d = fn(torch.from_numpy(x).to(dev), pow2=pow2)
            rq, rd = fo.f8_quantize_ref(x, rows, pow2)
            assert np.array_equal(d.cpu().numpy(), rd, equal_nan=True)
            assert np.array_equal(q.view(torch.uint8).cpu().numpy(), rq)


def test_quantize_writes_its_rows_only(q8):
    lib, torch, dev = q8
    x = torch.randn(5, 160, device=dev)
    q = torch.full((8, 160), 0x55, dtype=torch.uint8, device=dev)
    d = torch.full((8, 2), 9.0, device=dev)
    lib.f8_quantize_act(x, q=q[:5], d=d[:5])
    assert (q[5:] == 0x55).all() and (d[5:] == 9).all()
    assert torch.equal(q[:5], lib.f8_quantize_act(x)[0].view(torch.uint8))
    lib.f8_quantize_act(torch.empty(0, 160, device=dev))
    lib.f8_quantize_weight(torch.empty(0, 160, device=dev))


# ---------------------------------------------------------------------------- products

SHAPES = [(1, 1, 16), (1, 257, 1040), (1, 640, 4096), (2, 130, 128), (5, 48, 384), (16, 300, 2064), (17, 128, 272),
          (31, 1000, 512), (33, 515, 144), (64, 257, 1024), (65, 129, 640), (127, 384, 2048), (129, 2001, 1040),
          (200, 96, 4096), (257, 513, 656), (300, 1100, 256), (1030, 700, 384)]


def operands(q8, seed, m, n, k, parts=1):
    lib, torch, dev = q8
    rng = np.random.default_rng(seed)
    wq, wd, w = weight(rng, n, k, parts)
    xq, xd, x = inputs(rng, m, k)
    return to_dev(torch, dev, wq, wd, xq, xd), w, x


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear(q8, m, n, k, kind):
    lib, torch, dev = q8
    say(f"f8_linear m={m} n={n} k={k} {kind}")
    args, w, x = operands(q8, m + n + k, m, n, k)
    y = lib.f8_linear(*args, dtype=getattr(torch, kind))
    check(y, *product_limits(x, w, half_step(torch, kind)), f"f8_linear m={m} n={n} k={k} {kind}")


def activated(gu, worst, usual, half):
    """h and its limits: |SiLU'| <= 1.1; the activation's own exp, sum, quotient and product (|g| + 8) u each twice."""
    f = gu.shape[1] // 2
    g, u = gu[:, :f], gu[:, f:]
    s = g / (1 + np.exp(-g))
    h = s * u
    own = 2 * U * (np.abs(g) + 8) * np.abs(h)

    def limit(e):
        return 1.1 * np.abs(u) * e[:, :f] + np.abs(s) * e[:, f:] + 1.1 * e[:, :f] * e[:, f:] + own
    return h, limit(worst) + rounding(half, np.abs(h) + limit(worst)), limit(usual) + rounding(half, np.abs(h))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,f,k", SHAPES)
def test_gate_up(q8, m, f, k, kind):
    lib, torch, dev = q8
    say(f"f8 gate_up m={m} f={f} k={k} {kind}")
    args, w, x = operands(q8, m + f + k + 1, m, f, k, parts=2)
    half = half_step(torch, kind)
    h, gu = lib.f8_linear_fused_gate_up_silu(*args, dtype=getattr(torch, kind), keep_gate_up=True)
    check(gu, *product_limits(x, w, half), f"gate and up m={m} f={f} k={k} {kind}")
    check(h, *activated(*product_limits(x, w, 0.0, kind == "float32"), half), f"h m={m} f={f} k={k} {kind}")
    alone = lib.f8_linear_fused_gate_up_silu(*args, dtype=getattr(torch, kind))
    assert torch.equal(alone, h)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_exact_sums(q8, m, n, k):
    """Small whole numbers and scales that are powers of two: every sum is exact in float32."""
    lib, torch, dev = q8
    say(f"exact m={m} n={n} k={k}")
    rng = np.random.default_rng(m * 7 + n)
    wv, xv = rng.integers(-4, 5, (n, k)), rng.integers(-4, 5, (m, k))
    kb, nb = -(-k // 128), -(-n // 128)
    wd = 2.0 ** rng.integers(-1, 2, (nb, kb))
    xd = 2.0 ** rng.integers(-1, 2, (m, kb))
    wq, xq = fo.e4m3_encode(wv), fo.e4m3_encode(xv)
    w, x = fo.f8_values(wq, wd, 128), fo.f8_values(xq, xd, 1)
    args = to_dev(torch, dev, wq, wd.astype(np.float32), xq, xd.astype(np.float32))
    assert np.array_equal(lib.f8_linear(*args).cpu().numpy(), x @ w.T)
    # the 8-bit matrix cores hold these products whole: the result is the exact one rounded once
    want = torch.from_numpy(x @ w.T).float()
    for dtype in (torch.float16, torch.bfloat16):
        assert torch.equal(lib.f8_linear(*args, dtype=dtype).cpu(), want.to(dtype))


@pytest.mark.parametrize("m,n,k", [(2000, 6131, 400), (1793, 6001, 112), (4097, 6140, 128)])
def test_products_whose_rows_cross_blocks(q8, m, n, k):
    """Sizes between whole rounds of the largest tiles: waves of 48 weight rows, in two blocks of scales."""
    test_exact_sums(q8, m, n, k)
    for kind in ("bfloat16", "float16"):
        test_linear(q8, m, n, k, kind)


def test_every_code(q8):
    """Each of the 254 finite codes of either operand at its value, in every block position."""
    lib, torch, dev = q8
    codes = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    eye = np.zeros((128, 128), np.uint8)
    np.fill_diagonal(eye, 0x38)  # ones
    one = np.ones((1, 1), np.float32)
    for part in (codes[:127], codes[127:]):
        col = np.concatenate([part, part[:1]])[:, None].repeat(128, axis=1)
        args = to_dev(torch, dev, eye, one, col, np.ones((128, 1), np.float32))
        assert np.array_equal(lib.f8_linear(*args).cpu().numpy(), fo.e4m3_table()[col])
        args = to_dev(torch, dev, col, one, eye, np.ones((128, 1), np.float32))
        assert np.array_equal(lib.f8_linear(*args).cpu().numpy(), fo.e4m3_table()[col].T)


@pytest.mark.parametrize("m", [1, 9, 40, 130, 300])
def test_not_finite_stays_in_its_place(q8, m):
    lib, torch, dev = q8
    n, k = 300, 400
    (wq, wd, xq, xd), w, x = operands(q8, m, m, n, k)
    clean = lib.f8_linear(wq, wd, xq, xd)
    t = m // 2
    bad = xd.clone()
    bad[t, 3] = float("nan")
    y = lib.f8_linear(wq, wd, xq, bad)
    assert torch.isnan(y[t]).all() and torch.equal(y[:t], clean[:t]) and torch.equal(y[t + 1:], clean[t + 1:])
    codes = wq.clone()
    codes[299, 399] = 0x7F
    y = lib.f8_linear(codes, wd, xq, xd)
    assert torch.isnan(y[:, 299]).all() and torch.equal(y[:, :299], clean[:, :299])
    scales = wd.clone()
    scales[1, 0] = float("inf")
    y = lib.f8_linear(wq, scales, xq, xd)
    assert not torch.isfinite(y[:, 128:256]).any()
    assert torch.equal(y[:, :128], clean[:, :128]) and torch.equal(y[:, 256:], clean[:, 256:])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k", [(1, 70, 272), (40, 130, 512), (300, 261, 144)])
def test_strided_outputs(q8, m, n, k, kind):
    """Rows of any leading dimension and alignment; nothing outside them is written."""
    lib, torch, dev = q8
    args, _, _ = operands(q8, 5, m, n, k)
    dtype = getattr(torch, kind)
    want = lib.f8_linear(*args, dtype=dtype)
    for lead, shift in ((n + 3, 1), (n + 8, 0), (n, 0)):
        flat = torch.full((m * lead + 16,), -7.0, dtype=dtype, device=dev)
        out = flat[shift:shift + m * lead].view(m, lead)[:, :n]
        assert lib.f8_linear(*args, out=out) is out
        assert torch.equal(out, want)
        left = torch.ones_like(flat, dtype=torch.bool)
        left[shift:shift + m * lead].view(m, lead)[:, :n] = False
        assert (flat[left] == -7).all()
    args, _, _ = operands(q8, 6, m, n, k, parts=2)
    h, gu = lib.f8_linear_fused_gate_up_silu(*args, dtype=dtype, keep_gate_up=True)
    flat = torch.full((m * (2 * n + 5) + 1,), -7.0, dtype=dtype, device=dev)
    keep = flat[1:].view(m, 2 * n + 5)[:, :2 * n]
    h2, gu2 = lib.f8_linear_fused_gate_up_silu(*args, dtype=dtype, keep_gate_up=keep)
    assert gu2 is keep and torch.equal(gu2, gu) and torch.equal(h2, h) and (flat[1:].view(m, -1)[:, 2 * n:] == -7).all()


def test_nothing_to_do(q8):
    lib, torch, dev = q8
    (wq, wd, xq, xd), _, _ = operands(q8, 7, 4, 20, 160)
    assert lib.f8_linear(wq, wd, xq[:0], xd[:0]).shape == (0, 20)
    assert lib.f8_linear(wq[:0], wd[:0], xq, xd).shape == (4, 0)
    h, gu = lib.f8_linear_fused_gate_up_silu(wq, wd.repeat(2, 1), xq[:0], xd[:0], keep_gate_up=True)
    assert h.shape == (0, 10) and gu.shape == (0, 20)


def test_refusals(q8):
    lib, torch, dev = q8
    (wq, wd, xq, xd), _, _ = operands(q8, 8, 4, 20, 160)
    for bad in ((wq.float(), wd, xq, xd), (wq, wd.double(), xq, xd), (wq, wd[:, :1], xq, xd), (wq, wd, xq[:, :144], xd),
                (wq, wd, xq, xd[:3]), (wq.cpu(), wd, xq, xd), (wq.t(), wd, xq, xd), (wq, wd, xq, xd.t())):
        with pytest.raises(ValueError):
            lib.f8_linear(*bad)
    with pytest.raises(ValueError):
        lib.f8_linear(wq, wd, xq, xd, dtype=torch.float64)
    with pytest.raises(ValueError):
        lib.f8_linear(wq, wd, xq, xd, out=torch.empty(4, 21, device=dev))
    with pytest.raises(ValueError):
        lib.f8_linear_fused_gate_up_silu(wq, wd, xq, xd)  # scales of one matrix of 20 rows
    with pytest.raises(ValueError):
        lib.f8_linear_fused_gate_up_silu(wq[:19], wd, xq, xd)
    with pytest.raises(ValueError):
        lib.f8_quantize_act(torch.zeros(4, 16, dtype=torch.float64, device=dev))
    with pytest.raises(lib.Q8Error):
        lib.f8_quantize_act(torch.zeros(4, 24, device=dev))
    with pytest.raises(lib.Q8Error):
        lib.f8_quantize_act(torch.zeros(4, 35, device=dev)[:, :32])  # rows of 140 bytes
    with pytest.raises(lib.Q8Error):
        lib.f8_quantize_act(torch.zeros(4 * 16 + 1, device=dev)[1:].view(4, 16))


def test_repeats_streams_and_graphs(q8):
    """Same bits on every call, on a stream of its own, and in a replayed graph with changing inputs."""
    lib, torch, dev = q8
    for m in (1, 40, 300):
        (wq, wd, xq, xd), _, _ = operands(q8, 9 + m, m, 200, 784, parts=2)
        want = lib.f8_linear_fused_gate_up_silu(wq, wd, xq, xd, dtype=torch.bfloat16)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = lib.f8_linear_fused_gate_up_silu(wq, wd, xq, xd, dtype=torch.bfloat16)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, want)
        x = torch.randn(m, 784, device=dev)
        q, d = lib.f8_quantize_act(x)
        out = torch.empty(m, 200, dtype=torch.bfloat16, device=dev)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lib.f8_quantize_act(x, q=q, d=d)
            lib.f8_linear_fused_gate_up_silu(wq, wd, q, d, out=out)
        for turn in range(4):
            x.copy_(torch.randn(m, 784, device=dev))
            graph.replay()
            torch.cuda.synchronize()
            eager = lib.f8_linear_fused_gate_up_silu(wq, wd, *lib.f8_quantize_act(x), dtype=torch.bfloat16)
            assert torch.equal(out, eager), turn
