"""The 8-bit floating-point operators put together as a feed-forward block uses them, side by side on
streams and in graphs, and at sizes whose offsets pass 31 and 32 bits."""

from __future__ import annotations

import numpy as np
import pytest

import oracle.f8_oracle as fo
from f8_cases import U, floats, to_dev
from gpu_util import say, torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


class Block:
    """A gated feed-forward block with e4m3 weights, its forward pass and its gradients."""

    def __init__(self, q8, seed, k, f):
        self.lib, self.torch, self.dev = q8
        rng = np.random.default_rng(seed)
        gate, up, down = (to_dev(self.torch, self.dev, 0.05 * floats(rng, *s))[0] for s in ((f, k), (f, k), (k, f)))
        parts = [self.lib.f8_quantize_weight(w) for w in (gate, up)]
        self.gate_up = (self.torch.cat([q.view(self.torch.uint8) for q, _ in parts]), self.torch.cat([d for _, d in parts]))
        self.down = self.lib.f8_quantize_weight(down)

    def forward(self, x, dtype):
        lib = self.lib
        x8 = lib.f8_quantize_act(x)
        h, gu = lib.f8_linear_fused_gate_up_silu(*self.gate_up, *x8, dtype=dtype, keep_gate_up=True)
        h8 = lib.f8_quantize_act(h)
        return lib.f8_linear(*self.down, *h8, dtype=dtype), (x8, gu, h8)

    def backward(self, kept, dy):
        x8, gu, h8 = kept
        dh, d_down = self.lib.f8_linear_backward(*self.down, *h8, dy)
        dx, d_gate_up = self.lib.f8_linear_fused_gate_up_silu_backward(*self.gate_up, *x8, gu, dh)
        return dx, d_gate_up, d_down


def host(t, torch):
    codes = t.dtype in (torch.float8_e4m3fn, torch.uint8)
    return t.view(torch.uint8).cpu().numpy() if codes else t.double().cpu().numpy()


@pytest.mark.parametrize("m,k,f", [(1, 256, 80), (37, 400, 208), (300, 272, 528)])
def test_training_step(q8, m, k, f):
    """Forward and gradients in float32 against the formulas in float64 at the values that the calls kept."""
    lib, torch, dev = q8
    say(f"block m={m} k={k} f={f}")
    b = Block(q8, m, k, f)
    rng = np.random.default_rng(m + 1)
    x, dy = to_dev(torch, dev, floats(rng, m, k), floats(rng, m, k))
    y, kept = b.forward(x, torch.float32)
    dx, d_gate_up, d_down = b.backward(kept, dy)
    x8, gu, h8 = kept
    w1 = fo.f8_weight_values(host(b.gate_up[0], torch), host(b.gate_up[1], torch), 2)
    w2 = fo.f8_values(host(b.down[0], torch), host(b.down[1], torch), 128)
    xv = fo.f8_values(host(x8[0], torch), host(x8[1], torch), 1)
    hv = fo.f8_values(host(h8[0], torch), host(h8[1], torch), 1)
    guv, dyv = host(gu, torch), host(dy, torch)
    dh = dyv @ w2
    d = fo.f8_gate_up_gradient_ref(guv, dh)
    # every one a float32 product of at most max(m, k, 2f) terms, at worst behind another and an activation. A sum
    # of n roundings of random sign is off by 2^-24 sqrt(n) of its size; twice that, for either product
    limit = 4 * U * np.sqrt(max(m, k, 2 * f))
    for name, got, want in (("gu", guv, xv @ w1.T), ("y", host(y, torch), hv @ w2.T), ("d_down", host(d_down, torch), dyv.T @ hv),
                            ("dx", host(dx, torch), d @ w1), ("d_gate_up", host(d_gate_up, torch), d.T @ xv)):
        off = np.linalg.norm(got - want) / np.linalg.norm(want)
        say(f"{name}: {off:.1e} of {limit:.1e}")
        assert off <= limit, name
    # what the next product reads is the rounded activation: within half a step of e4m3 and of its scale
    act = fo.f8_gate_up_ref(guv)
    assert (np.abs(hv - act) <= 2.0 ** -4 * np.abs(act) + 2.0 ** -9 * host(h8[1], torch).repeat(128, axis=1)[:, :f]).all()


def test_steps_beside_each_other(q8):
    """Two blocks' steps on two streams at once, each with the bits that it has alone."""
    lib, torch, dev = q8
    blocks = [Block(q8, s, 512, 384) for s in (1, 2)]
    xs = [torch.randn(200, 512, device=dev) for _ in blocks]
    dys = [torch.randn(200, 512, device=dev).bfloat16() for _ in blocks]

    def step(b, x, dy):
        y, kept = b.forward(x, torch.bfloat16)
        return (y, *b.backward(kept, dy))

    alone = [step(b, x, dy) for b, x, dy in zip(blocks, xs, dys)]
    streams = [torch.cuda.Stream() for _ in blocks]
    torch.cuda.synchronize()
    beside = []
    for turn in range(3):
        for s, b, x, dy in zip(streams, blocks, xs, dys):
            with torch.cuda.stream(s):
                beside.append(step(b, x, dy))
    torch.cuda.synchronize()
    for i, got in enumerate(beside):
        assert all(torch.equal(a, c) for a, c in zip(got, alone[i % 2])), i


def test_captured_step(q8):
    """A whole step in a graph, replayed between eager steps of the same block."""
    lib, torch, dev = q8
    b = Block(q8, 3, 400, 272)
    x, dy = torch.randn(150, 400, device=dev), torch.randn(150, 400, device=dev).bfloat16()

    def step():
        y, kept = b.forward(x, torch.bfloat16)
        return (y, *b.backward(kept, dy))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for turn in range(4):
        x.copy_(torch.randn(150, 400, device=dev))
        dy.copy_(torch.randn(150, 400, device=dev))
        graph.replay()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), turn


# ------------------------------------------------------------------ offsets past 31 and 32 bits


def few(torch, dev, rows, k, seed):
    """Codes 0 and +-1 on the device, a few ones a row, and scales of one."""
    gen = torch.Generator(device=dev).manual_seed(seed)
    q = torch.zeros(rows, k, dtype=torch.uint8, device=dev)
    at = torch.randint(0, k, (rows, 8), generator=gen, device=dev)
    sign = torch.randint(0, 2, (rows, 8), generator=gen, device=dev).to(torch.uint8) * 0x80 + 0x38
    q.scatter_(1, at, sign)
    return q


def value(torch, q):
    return q.view(torch.float8_e4m3fn).float()


@pytest.mark.parametrize("m", [5, 100, 400])
def test_large_matrix(q8, m):
    """W of more than 2^32 bytes: the rows behind its ends are multiplied right."""
    lib, torch, dev = q8
    n, k = (1 << 18) + 77, 16 * 1033
    say(f"large matrix {n} x {k}, {m} rows")
    w, x = few(torch, dev, n, k, 1), few(torch, dev, m, k, 2)
    wd = torch.ones(-(-n // 128), -(-k // 128), device=dev)
    xd = torch.ones(m, -(-k // 128), device=dev)
    y = lib.f8_linear(w, wd, x, xd, dtype=torch.bfloat16)
    rows = torch.tensor([0, 1, 4095, 131071, 131072, 200000, n - 129, n - 128, n - 1], device=dev)
    want = value(torch, x) @ value(torch, w[rows]).T
    assert torch.equal(y[:, rows].float(), want)
    f = n // 2
    h, gu = lib.f8_linear_fused_gate_up_silu(w[:2 * f], torch.ones(2 * -(-f // 128), wd.shape[1], device=dev), x, xd,
                                             dtype=torch.bfloat16, keep_gate_up=True)
    rows = rows[rows < 2 * f]
    assert torch.equal(gu[:, rows].float(), value(torch, x) @ value(torch, w[rows]).T)


def test_large_batch(q8):
    """Activations, gradients and planes of more than 2^32 bytes."""
    lib, torch, dev = q8
    m, n, k = (1 << 18) + 77, 40, 16 * 1033
    say(f"large batch of {m} rows of {k}")
    w, x = few(torch, dev, n, k, 3), few(torch, dev, m, k, 4)
    wd = torch.ones(1, -(-k // 128), device=dev)
    xd = torch.ones(m, -(-k // 128), device=dev)
    rows = torch.tensor([0, 130000, 131072, 259999, m - 257, m - 1], device=dev)
    y = lib.f8_linear(w, wd, x, xd)
    assert torch.equal(y[rows], value(torch, x[rows]) @ value(torch, w).T)
    del y
    dy = torch.zeros(m, n, dtype=torch.bfloat16, device=dev)
    dy[rows] = torch.randint(-2, 3, (len(rows), n), device=dev).bfloat16()
    dx, dw = lib.f8_linear_backward(w, wd, x, xd, dy)
    assert torch.equal(dx[rows].float(), dy[rows].float() @ value(torch, w))
    assert torch.equal(dw.float(), dy[rows].float().T @ value(torch, x[rows]))
    del dx, dw
    q, d = lib.f8_quantize_act(value(torch, x[-70000:]).bfloat16(), pow2=True)
    assert (d[:, -1] <= 2.0 ** -8).all() and torch.equal(value(torch, q) * d.repeat_interleave(128, 1)[:, :k], value(torch, x[-70000:]))


def test_refuses_what_is_no_tensor(q8):
    """Operands and outputs that are not tensors: a ValueError, as for every wrong one."""
    lib, torch, dev = q8
    x, w = torch.ones(3, 256, device=dev), torch.ones(130, 256, device=dev)
    (xq, xd), (wq, wd) = lib.f8_quantize_act(x), lib.f8_quantize_weight(w)
    calls = (lambda: lib.f8_quantize_act(x, q=[0]), lambda: lib.f8_quantize_act(x, d=[0.0]),
             lambda: lib.f8_quantize_weight(w, q=7), lambda: lib.f8_linear(wq, wd, xq, xd, out=[1.0]),
             lambda: lib.f8_linear_fused_gate_up_silu(wq, wd, xq, xd, out=1),
             lambda: lib.f8_linear(wq, None, xq, xd), lambda: lib.f8_linear(wq, wd, [1], xd),
             lambda: lib.f8_linear_backward(wq, wd, xq, xd, [1.0]))
    for call in calls:
        with pytest.raises(ValueError):
            call()
