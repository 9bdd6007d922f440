"""q8_moe_layer routes like moe_route_topk: the same experts, order and weights, bit for bit.

The layer does not return its choice, so the experts here make it visible.  With x[t][0] = 1
every expert's only hidden element is SiLU(64) * 1 = 64 (1 + exp(-64) is 1 in float32), and
expert e's down projection puts it into output e alone: y[t][e] = 64 w, w the weight that
token t gives expert e (0 where it does not choose it).  Every step is exact, powers of two
times w."""

from __future__ import annotations

import numpy as np
import pytest

import workloads as wl
from gpu_util import say, to_dev, torch_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


def visible_experts(torch, dev, e, f, h):
    """(gate_up, down): Q8_0 stacks whose blocks of scale 1 hold one quant each."""
    one = torch.tensor([0x00, 0x3C], dtype=torch.uint8, device=dev)  # binary16 1.0
    gu = torch.zeros((e, 2 * f, h // 32, 34), dtype=torch.uint8, device=dev)
    gu[:, 0, 0, :2], gu[:, 0, 0, 2] = one, 64
    gu[:, f, 0, :2], gu[:, f, 0, 2] = one, 1
    dn = torch.zeros((e, h, f // 32, 34), dtype=torch.uint8, device=dev)
    ids = torch.arange(e, device=dev)
    dn[ids, ids, 0, :2], dn[ids, ids, 0, 2] = one, 1
    return gu.view(-1), dn.view(-1)


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("m,e,k,h", [(64, 128, 8, 2048), (128, 128, 7, 512), (128, 256, 15, 256), (31, 256, 64, 256),
                                     (15, 128, 64, 1280), (60, 60, 4, 768), (23, 3, 1, 256), (3, 5, 5, 256),
                                     (7, 1, 1, 256), (1, 200, 33, 4096)])
def test_the_layer_chooses_as_the_routers(q8, m, e, k, h, normalize):
    lib, torch, dev = q8
    f = 256
    gu, dn = visible_experts(torch, dev, e, f, h)
    x = wl.activations(4100 + m + e, m, h)
    x[:, 0] = 1.0
    xd, wr = to_dev(x, dev), to_dev(wl.router_weight(4200 + e, e, h, 0.05), dev)
    for top_p in (None, 0.9, 0.5):
        idx, w = lib.moe_route_topk(xd, wr, k, normalize, top_p=top_p)
        want = torch.zeros((m, e + 1), device=dev)
        want.scatter_(1, torch.where(idx < 0, e, idx).long(), w)  # dropped slots behind the experts
        y = lib.q8_moe_layer(wr, gu, dn, e, f, h, xd, k, normalize=normalize, top_p=top_p)
        got, want = y[:, :e] / 64, want[:, :e]
        off = int((got != want).any(dim=1).sum())
        say(f"m={m} e={e} k={k} h={h} normalize={normalize} top_p={top_p}: {off} tokens differ, "
            f"largest {float((got - want).abs().max()):.1e}")
        assert torch.equal(got, want) and not y[:, e:].any()
        assert torch.equal((got != 0), (want != 0))


def test_the_layer_chooses_as_the_routers_among_equals(q8):
    """Equal logits (the lowest experts win), and a cut at the exact share."""
    lib, torch, dev = q8
    m, e, k, f, h = 5, 160, 6, 256, 256
    gu, dn = visible_experts(torch, dev, e, f, h)
    x = np.zeros((m, h), np.float32)
    x[:, 0] = 1.0
    wr = np.zeros((e, h), np.float32)
    wr[[3, 70, 130, 159], 0] = 1.0  # four share the largest logit, in three planes of 64
    xd, wrd = to_dev(x, dev), to_dev(wr, dev)
    for top_p in (None, 0.25, 0.5, 1.0):
        idx, w = lib.moe_route_topk(xd, wrd, k, True, top_p=top_p)
        want = torch.zeros((m, e + 1), device=dev)
        want.scatter_(1, torch.where(idx < 0, e, idx).long(), w)
        y = lib.q8_moe_layer(wrd, gu, dn, e, f, h, xd, k, top_p=top_p)
        assert torch.equal(y[:, :e] / 64, want[:, :e]), top_p
