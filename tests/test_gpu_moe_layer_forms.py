"""Forms of q8_moe_layer at their limits: many experts a token, the largest pair lists, the
first sizes past the two-launch form, tokens that are not finite in the separate calls, and
several calls on the device at once."""

from __future__ import annotations

import numpy as np
import pytest

import oracle
import workloads as wl
from gpu_util import say, to_dev, torch_dev
from test_gpu_moe_layer import check, layer, mixture

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


# float32 range: m * k < 8 * experts.  More than eight experts a token (9, 17), a lane each (64) and one
# more than that (65: the separate calls); 128 tokens and 129 (the separate calls); 2047 pairs, the most there
# are, and 1920 in tokens of 15
@pytest.mark.parametrize("m,e,k,f,h", [(7, 40, 9, 256, 256), (20, 64, 17, 256, 512), (15, 128, 64, 256, 256),
                                       (15, 128, 65, 256, 256), (128, 128, 7, 256, 256), (129, 128, 7, 256, 256),
                                       (89, 256, 23, 256, 256), (128, 256, 15, 256, 256)])
def test_layer_at_its_limits(q8, m, e, k, f, h):
    lib, torch, dev = q8
    say(f"moe layer m={m} e={e} k={k} f={f} h={h}")
    gu, dn, wr = layer(5000 + 7 * m + e, e, f, h)
    x = wl.activations(5001 + m, m, h)
    args = (to_dev(wr, dev), to_dev(gu, dev), to_dev(dn, dev), e, f, h, to_dev(x, dev), k)
    for normalize, top_p in ((True, None), (False, 0.7)):
        y = lib.q8_moe_layer(*args, normalize=normalize, top_p=top_p)
        idx, _ = lib.moe_route_topk(args[6], args[0], k, normalize, top_p=top_p)
        idx = idx.cpu().numpy()
        p = oracle.softmax_ref(oracle.router_logits_ref(x, wr))
        wts = np.where(idx >= 0, np.take_along_axis(p, np.maximum(idx, 0).astype(np.int64), axis=1), 0.0)
        if normalize:
            wts = wts / wts.sum(axis=1, keepdims=True)
        check(y, *mixture(gu, dn, wr, e, f, h, x, idx, wts), f"normalize={normalize} top_p={top_p}")


# bf16 tiles from 8 pairs an expert on; past 128 tokens, 64 experts a token and width 6144 in float32
@pytest.mark.parametrize("top_p", [None, 0.6])
@pytest.mark.parametrize("m,e,k,f,h", [(70, 16, 2, 256, 512), (130, 128, 2, 256, 256), (9, 128, 65, 256, 256),
                                       (6, 4, 2, 256, 6400)])
def test_tokens_that_are_not_finite_in_the_separate_calls(q8, m, e, k, f, h, top_p):
    """NaN, whole; the others are what the routing and the grouped call give."""
    lib, torch, dev = q8
    gu, dn, wr = (to_dev(v, dev) for v in layer(5200, e, f, h))
    x = to_dev(wl.activations(5201, m, h), dev)
    x[0, 3], x[2, h - 1], x[m - 1, 0] = float("nan"), float("inf"), float("-inf")
    y = lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k, top_p=top_p)
    bad = [0, 2, m - 1]
    keep = [t for t in range(m) if t not in bad]
    assert torch.isnan(y[bad]).all()
    idx, w = lib.moe_route_topk(x, wr, k, True, top_p=top_p)
    two = lib.q8_moe_grouped_linear(gu, dn, e, f, h, x, idx, w)
    assert torch.isfinite(two[keep]).all() and torch.equal(y[keep], two[keep])


def test_four_calls_at_once(q8):
    """A block of the layer fills a compute unit, so the blocks of four calls on four streams
    wait for one another: what a late block would have worked on, those that are there take
    over.  Every call gives the bits of a call alone."""
    lib, torch, dev = q8
    e, k, f, h = 64, 8, 512, 1024
    gu, dn, wr = (to_dev(v, dev) for v in layer(5300, e, f, h))
    sizes = (1, 60, 17, 33)
    xs = [to_dev(wl.activations(5301 + m, m, h), dev) for m in sizes]
    want = [lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k) for x in xs]
    ws = [torch.empty(lib.q8_moe_layer_workspace_bytes(m, k, e, f, h), dtype=torch.uint8, device=dev) for m in sizes]
    streams = [torch.cuda.Stream() for _ in sizes]
    torch.cuda.synchronize()
    outs = [[torch.full((m, h), float("nan"), device=dev) for m in sizes] for _ in range(8)]
    torch.cuda.synchronize()
    for r in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                lib.q8_moe_layer(wr, gu, dn, e, f, h, xs[i], k, out=outs[r][i], workspace=ws[i])
    torch.cuda.synchronize()
    for r in range(8):
        for i in range(4):
            assert torch.equal(outs[r][i], want[i]), (r, i)
