"""The adapter calls and the MoE layer at sizes where offsets and grids pass 31 and 32 bits,
against the framework's other calls on the same data."""

from __future__ import annotations

import pytest

from gpu_util import say, torch_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    yield q8mod, torch, dev
    torch.cuda.empty_cache()


def packed(torch, dev, rows, k, seed):
    """Q8_0 bytes: any quants, scales of 2^-9."""
    gen = torch.Generator(device=dev).manual_seed(seed)
    w = torch.randint(0, 256, (rows, k // 32, 34), dtype=torch.uint8, device=dev, generator=gen)
    w[:, :, 0], w[:, :, 1] = 0, 0x18
    return w.view(-1)


def adapters(torch, dev, m, n, k, sections, seed):
    gen = torch.Generator(device=dev).manual_seed(seed)
    a = torch.randn((2, len(sections) * 8, k), generator=gen, device=dev) / k ** 0.5
    b = torch.randn((2, n, 8), generator=gen, device=dev)
    ids = torch.tensor([1, -1, 0, 1], dtype=torch.int32, device=dev)[:m]
    return (a, b, ids), dict(sections=sections), torch.randn((m, k), generator=gen, device=dev)


def off(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


# rows of 4352 bytes: 493,440 of them end 32 KB below 2 GiB (digit tiles, two rows and more),
# 493,504 pass it (the packed linear's kernels, then the correction)
@pytest.mark.parametrize("n,m", [(493440, 4), (493440, 1), (493504, 4), (493504, 1)])
def test_matrices_about_2_gib(q8, n, m):
    lib, torch, dev = q8
    k, f = 4096, n // 2
    w = packed(torch, dev, n, k, 1)
    assert (w.numel() < 2 ** 31) == (n == 493440)
    args, more, x = adapters(torch, dev, m, n, k, [f, f], 2)
    # both products are of float32 accuracy: sqrt(k / 32 + 52) roundings and 8 more each, as
    # sums of random terms; the correction's products add at most 16 + sqrt(k / 8 + 28)
    tol = U * (2 * ((k / 32 + 52) ** 0.5 + 8) + 16 + (k / 8 + 28) ** 0.5)
    want = lib.lora_add(lib.q8_linear(w, n, k, x), x, *args, **more)
    got = lib.q8_linear_lora(w, n, k, x, *args, **more)
    say(f"n={n} m={m}: {off(got, want):.1e}, at most {tol:.1e}")
    assert off(got, want) <= tol and off(got[:, -64:], want[:, -64:]) <= tol
    h = lib.q8_linear_fused_gate_up_silu_lora(w, f, k, x, *args, **more)
    g, u = want[:, :f].double(), want[:, f:].double()
    # |SiLU'| <= 1.1, and the rounding of the activation
    limit = (1.1 * u.abs() * tol * g.norm() / g.numel() ** 0.5 + (g * torch.sigmoid(g)).abs() * tol * u.norm() / u.numel() ** 0.5
             + (g.abs() + 8) * 2 * U * (g * torch.sigmoid(g) * u).abs()).norm()
    assert float((h.double() - g * torch.sigmoid(g) * u).norm()) <= float(limit)


def test_more_threads_than_32_bits_hold(q8):
    """700 rows of 2^23 outputs: an output a thread is 5.9 billion of them."""
    lib, torch, dev = q8
    m, n, k, rank, count = 700, 1 << 23, 256, 8, 256
    a = torch.ones((count, rank, k), dtype=torch.bfloat16, device=dev)
    b = torch.zeros((count, n, rank), dtype=torch.bfloat16, device=dev)
    b[7, -5:], b[187, :3] = 0.25, 0.5
    x = torch.ones((m, k), device=dev)
    ids = (torch.arange(m, device=dev) % count).int()
    y = torch.zeros((m, n), device=dev)
    assert lib.lora_add(y, x, a, b, ids, out=y) is y
    last, first = torch.where(ids == 7, rank * k * 0.25, 0.0), torch.where(ids == 187, rank * k * 0.5, 0.0)
    assert torch.equal(y[:, -5:], last[:, None].expand(m, 5)) and torch.equal(y[:, :3], first[:, None].expand(m, 3))
    assert not y[:, 3:-5].any()


def test_expert_stacks_past_32_bits(q8):
    """256 experts of 2048 x 4096 (4.6 GB of gate and up rows): against routing and mixture."""
    lib, torch, dev = q8
    e, k, f, h, m = 256, 4, 2048, 4096, 40
    gu, dn = packed(torch, dev, e * 2 * f, h, 3), packed(torch, dev, e * h, f, 4)
    assert gu.numel() > 2 ** 32
    gen = torch.Generator(device=dev).manual_seed(5)
    x = torch.randn((m, h), generator=gen, device=dev)
    wr = torch.randn((e, h), generator=gen, device=dev) / h ** 0.5
    wr[e - 1] = x[0] / 32  # token 0 takes the last expert
    idx, w = lib.moe_route_topk(x, wr, k, True)
    assert int(idx[0, 0]) == e - 1 and int(idx.unique().numel()) > 64
    two = lib.q8_moe_grouped_linear(gu, dn, e, f, h, x, idx, w)
    got = lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k)
    # two products of float32 accuracy on both sides, SiLU between them (argument errors
    # times |g|: the gates here are of the size of 64 * 2^-9 * 74 * 4 = 37)
    tol = 2 * U * (2 * ((h / 32 + 52) ** 0.5 + 8) + 2 * 37 + 8)
    say(f"{off(got, two):.1e}, at most {tol:.1e}")
    assert off(got, two) <= tol and off(got[:1], two[:1]) <= tol
