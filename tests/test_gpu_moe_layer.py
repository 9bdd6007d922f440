"""GPU parity of q8_moe_layer against the oracle's routing and mixture in float64, and
against the library's own moe_route_topk and q8_moe_grouped_linear."""

from __future__ import annotations

import numpy as np
import pytest

import oracle
import workloads as wl
from gpu_util import assert_close, moe_mixture_grouped_ref, say, to_dev, torch_dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def gamma(d):
    return d * U / (1 - d * U)


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


def layer(seed, e, f, h, std=0.05):
    gu = np.concatenate([wl.q8_weight(seed + i, 2 * f, h)[0] for i in range(e)])
    dn = np.concatenate([wl.q8_weight(seed + 500 + i, h, f)[0] for i in range(e)])
    return gu, dn, wl.router_weight(seed + 999, e, h, std)


def mixture(gu, dn, wr, e, f, h, x, idx, wts):
    """(y, bound) in float64 for the given routing.  The bound follows the errors through the
    layer: a product of width w is off by gamma(w / 32 + 52) of its terms' magnitudes, and by
    2^-30 of its row's largest magnitude times the weights' (x may be taken as 32-bit fixed
    point); the activation as |SiLU'| <= 1.1 and its own (|g| + 8) 2^-23; the weights of the
    experts by twice the largest logit error (their softmax's) and k + 8 roundings; the final
    sum by k roundings."""
    m, k = idx.shape
    x = x.astype(np.float64)
    y, err = np.zeros((m, h)), np.zeros((m, h))
    gb, db = 2 * f * h // 32 * 34, h * f // 32 * 34
    logit = gamma(h // 64 + 8) * (np.abs(x) @ np.abs(wr.astype(np.float64)).T).max(axis=1)
    for i in range(e):
        t, j = np.nonzero(idx == i)
        if not t.size:
            continue
        w1 = oracle.dequantize_q8_0(gu[i * gb:(i + 1) * gb], 2 * f, h)
        w2 = oracle.dequantize_q8_0(dn[i * db:(i + 1) * db], h, f)
        xa = np.abs(x[t])
        v = x[t] @ w1.T
        ve = gamma(h / 32 + 52) * (xa @ np.abs(w1).T) + 2.0 ** -30 * xa.max(axis=1)[:, None] * np.abs(w1).sum(axis=1)
        g, u, ge, ue = v[:, :f], v[:, f:], ve[:, :f], ve[:, f:]
        s = oracle.silu_ref(g)
        hid = s * u
        he = 1.1 * ge * (np.abs(u) + ue) + np.abs(s) * ue + (np.abs(g) + 8) * 2.0 ** -23 * np.abs(hid)
        ha = np.abs(hid) + he
        o = hid @ w2.T
        oe = he @ np.abs(w2).T + gamma(f / 32 + 52) * (ha @ np.abs(w2).T)
        oe += 2.0 ** -30 * ha.max(axis=1)[:, None] * np.abs(w2).sum(axis=1)
        p = wts[t, j][:, None]
        np.add.at(y, t, p * o)
        np.add.at(err, t, p * (oe + (np.abs(o) + oe) * (2 * logit[t][:, None] + gamma(2 * k + 8))))
    return y, err


def check(got, want, bound, what):
    off = np.abs(got.cpu().numpy().astype(np.float64) - want)
    worst = float((off / np.maximum(bound, 1e-300)).max()) if off.size else 0.0
    say(f"{what}: worst error {worst:.4f} of its bound, rel {np.linalg.norm(off) / max(np.linalg.norm(want), 1e-300):.1e}")
    assert np.all(off <= bound), what


# m, experts, k, f, h: one token to many, one expert, all experts chosen, experts with more
# tokens than one pass takes, widths whose slices do not divide evenly among the waves
CASES = [(1, 8, 2, 256, 256), (1, 1, 1, 256, 512), (3, 5, 5, 512, 256), (5, 8, 2, 768, 2048), (7, 8, 2, 1792, 1280),
         (16, 16, 4, 256, 1024), (15, 2, 1, 256, 768), (13, 4, 2, 512, 1536), (2, 3, 3, 2048, 2304),
         (31, 64, 8, 256, 512), (100, 60, 4, 256, 256), (6, 4, 2, 256, 4096), (4, 3, 2, 3840, 512),
         (64, 256, 8, 256, 256), (200, 128, 3, 256, 256), (5, 2, 2, 4352, 256), (3, 2, 1, 256, 8448)]


@pytest.mark.parametrize("m,e,k,f,h", CASES)
def test_layer_vs_oracle(q8, m, e, k, f, h):
    lib, torch, dev = q8
    say(f"moe layer m={m} e={e} k={k} f={f} h={h}")
    gu, dn, wr = layer(3000 + 7 * m + e, e, f, h)
    x = wl.activations(3001 + m, m, h)
    args = (to_dev(wr, dev), to_dev(gu, dev), to_dev(dn, dev), e, f, h, to_dev(x, dev), k)
    for normalize, top_p in ((True, None), (False, 0.8)):
        y = lib.q8_moe_layer(*args, normalize=normalize, top_p=top_p)
        idx, _ = lib.moe_route_topk(args[6], args[0], k, normalize, top_p=top_p)
        idx = idx.cpu().numpy()
        # the library's own choice (its order is pinned by its own tests), the oracle's weights
        p = oracle.softmax_ref(oracle.router_logits_ref(x, wr))
        wts = np.where(idx >= 0, np.take_along_axis(p, np.maximum(idx, 0).astype(np.int64), axis=1), 0.0)
        if normalize:
            wts = wts / wts.sum(axis=1, keepdims=True)
        check(y, *mixture(gu, dn, wr, e, f, h, x, idx, wts), f"normalize={normalize} top_p={top_p}")


def test_a3b_layer(q8):
    """The Qwen3-30B-A3B layer, 16 tokens, against the oracle end to end."""
    lib, torch, dev = q8
    cfg = wl.QWEN3_30B_A3B_MOE
    gu, dn, wr = layer(cfg.seed * 10000, cfg.n_exp, cfg.ffn, cfg.hidden, cfg.router_std)
    x = wl.activations(cfg.seed + 1, cfg.tokens, cfg.hidden)
    xd, wrd, gud, dnd = (to_dev(v, dev) for v in (x, wr, gu, dn))
    y = lib.q8_moe_layer(wrd, gud, dnd, cfg.n_exp, cfg.ffn, cfg.hidden, xd, cfg.k)
    ridx, rw = oracle.route_topk_ref(x, wr, cfg.k, True)
    ref = moe_mixture_grouped_ref(gu, dn, cfg.n_exp, cfg.ffn, cfg.hidden, x, ridx, rw)
    assert_close(y.cpu().numpy(), ref, "a3b layer", tol=1e-5)
    idx, w = lib.moe_route_topk(xd, wrd, cfg.k, True)
    two = lib.q8_moe_grouped_linear(gud, dnd, cfg.n_exp, cfg.ffn, cfg.hidden, xd, idx, w)
    assert_close(y.cpu().numpy(), two.cpu().numpy(), "a3b layer against its two calls", tol=1e-5)
    for _ in range(5):
        assert torch.equal(y, lib.q8_moe_layer(wrd, gud, dnd, cfg.n_exp, cfg.ffn, cfg.hidden, xd, cfg.k))


def test_prefill_runs_the_grouped_tiles(q8):
    """From 8 routed pairs an expert on: the same bits as routing and the grouped call."""
    lib, torch, dev = q8
    m, e, k, f, h = 70, 8, 2, 256, 512
    gu, dn, wr = (to_dev(v, dev) for v in layer(3100, e, f, h))
    x = to_dev(wl.activations(3101, m, h), dev)
    idx, w = lib.moe_route_topk(x, wr, k, True)
    assert torch.equal(lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k),
                       lib.q8_moe_grouped_linear(gu, dn, e, f, h, x, idx, w))


@pytest.mark.parametrize("m", [6, 60])
def test_tokens_that_are_not_finite_stay_apart(q8, m):
    """Their outputs are NaN, whole; every other token's bits are those without them."""
    lib, torch, dev = q8
    e, k, f, h = 16, 2, 256, 512
    gu, dn, wr = (to_dev(v, dev) for v in layer(3200, e, f, h))
    x = to_dev(wl.activations(3201, m, h), dev)
    good = lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k)
    bad = x.clone()
    bad[0, 3], bad[2, 500], bad[5, 0] = float("nan"), float("inf"), float("-inf")
    y = lib.q8_moe_layer(wr, gu, dn, e, f, h, bad, k)
    keep = [t for t in range(m) if t not in (0, 2, 5)]
    assert torch.isnan(y[[0, 2, 5]]).all() and torch.equal(y[keep], good[keep])
    y = lib.q8_moe_layer(wr, gu, dn, e, f, h, torch.full_like(x, float("nan")), k)
    assert torch.isnan(y).all()


@pytest.mark.parametrize("e,k,f,h,most", [(16, 2, 256, 512, 63), (64, 8, 512, 1280, 60), (4, 3, 768, 256, 10)])
def test_a_token_depends_on_itself_alone(q8, e, k, f, h, most):
    """Any subset of the tokens gives the same bits, tokens alone included."""
    lib, torch, dev = q8
    gu, dn, wr = (to_dev(v, dev) for v in layer(3250, e, f, h))
    x = to_dev(wl.activations(3251, most, h), dev)
    whole = lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k)
    rng = np.random.default_rng(3252)
    for m in (1, 2, 3, 5, 8, 10):
        rows = torch.from_numpy(np.sort(rng.choice(most, m, replace=False))).to(dev)
        assert torch.equal(lib.q8_moe_layer(wr, gu, dn, e, f, h, x[rows].contiguous(), k), whole[rows]), m


def test_many_calls_in_a_row_on_one_workspace(q8):
    """Calls of changing sizes back to back on one workspace, none waited for."""
    lib, torch, dev = q8
    e, k, f, h = 32, 4, 256, 768
    gu, dn, wr = (to_dev(v, dev) for v in layer(3260, e, f, h))
    xs = [to_dev(wl.activations(3261 + m, m, h), dev) for m in (1, 33, 2, 60, 7)]
    ws = torch.empty(lib.q8_moe_layer_workspace_bytes(60, k, e, f, h), dtype=torch.uint8, device=dev)
    want = [lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k) for x in xs]
    got = [lib.q8_moe_layer(wr, gu, dn, e, f, h, xs[i % 5], k, workspace=ws) for i in range(40)]
    assert all(torch.equal(got[i], want[i % 5]) for i in range(40))


def test_zero_tokens_ties_and_zero_rows(q8):
    """No token; rows of zeros (every logit ties: the lowest experts; outputs 0)."""
    lib, torch, dev = q8
    e, k, f, h = 12, 3, 256, 256
    gu, dn, wr = (to_dev(v, dev) for v in layer(3300, e, f, h))
    assert lib.q8_moe_layer(wr, gu, dn, e, f, h, torch.empty((0, h), device=dev), k).shape == (0, h)
    x = torch.zeros((4, h), device=dev)
    x[1] = torch.randn(h, device=dev)
    y = lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k)
    assert (y[[0, 2, 3]] == 0).all()
    assert torch.equal(y[1:2], lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k)[1:2])


@pytest.mark.parametrize("m", [1, 9])
def test_strides_and_rows_behind_the_last(q8, m):
    lib, torch, dev = q8
    e, k, f, h = 8, 2, 256, 512
    gu, dn, wr = (to_dev(v, dev) for v in layer(3400, e, f, h))
    x = torch.full((m + 1, h + 4), float("nan"), device=dev)
    x[:m, :h] = to_dev(wl.activations(3401, m, h), dev)
    buf = torch.full((m + 2, h + 3), 7.0, device=dev)
    y = lib.q8_moe_layer(wr, gu, dn, e, f, h, x[:m, :h], k, out=buf[1:m + 1, :h])
    assert torch.equal(y.contiguous(), lib.q8_moe_layer(wr, gu, dn, e, f, h, x[:m, :h].contiguous(), k))
    assert (buf[0] == 7).all() and (buf[m + 1:] == 7).all() and (buf[:, h:] == 7).all()


def test_streams_workspaces_and_graphs(q8):
    """Calls on two streams at once with workspaces of their own, and captured calls
    replayed between eager ones, give the bits of a call alone, whatever the workspaces held."""
    lib, torch, dev = q8
    m, e, k, f, h = 12, 32, 4, 512, 1024
    gu, dn, wr = (to_dev(v, dev) for v in layer(3500, e, f, h))
    xs = [to_dev(wl.activations(3501 + i, m, h), dev) for i in range(2)]
    want = [lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k) for x in xs]
    size = lib.q8_moe_layer_workspace_bytes(m, k, e, f, h)
    ws = [torch.full((size,), 0xFF, dtype=torch.uint8, device=dev) for _ in range(3)]
    outs = [torch.empty((m, h), device=dev) for _ in range(2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                lib.q8_moe_layer(wr, gu, dn, e, f, h, xs[i], k, out=outs[i], workspace=ws[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    x = xs[0].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k, workspace=ws[2])
    for i in range(4):
        x.copy_(xs[i % 2])
        ws[2].fill_(17 * i)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i % 2]), i
        assert torch.equal(lib.q8_moe_layer(wr, gu, dn, e, f, h, xs[1], k), want[1])


def test_binding_refusals(q8):
    lib, torch, dev = q8
    e, k, f, h, m = 4, 2, 256, 256, 3
    gu, dn, wr = (to_dev(v, dev) for v in layer(3600, e, f, h))
    x = torch.zeros((m, h), device=dev)

    def call(err, wr=wr, gu=gu, dn=dn, x=x, k=k, **kw):
        with pytest.raises(err):
            lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k, **kw)

    call(ValueError, wr=wr[:3])
    call(ValueError, wr=wr.double())
    call(ValueError, gu=gu[:-1])
    call(ValueError, dn=dn[:-1])
    call(ValueError, x=x.half())
    call(ValueError, x=torch.zeros((m, h + 4), device=dev))
    call(ValueError, out=torch.empty((m, h - 1), device=dev))
    call(lib.Q8Error, k=5)
    call(lib.Q8Error, top_p=0.0)
    call(lib.Q8Error, top_p=1.5)
    call(lib.Q8Error, workspace=torch.empty(16, dtype=torch.uint8, device=dev))


def test_a_decode_step_together(q8):
    """The packed products of one decoder block as a serving step runs them: q/k/v with
    adapters, the output projection with adapters, then the MoE layer, on one stream."""
    lib, torch, dev = q8
    m, hid, e, k, f = 6, 512, 8, 2, 256
    rng = np.random.default_rng(3700)
    gu, dn, wr = layer(3701, e, f, hid)
    parts, x = [512, 256, 256], wl.activations(3702, m, hid)
    wq, wo = wl.q8_weight(3703, 1024, hid)[0], wl.q8_weight(3704, hid, 512)[0]
    aq, bq = rng.standard_normal((2, 24, hid)) / 22, 0.1 * rng.standard_normal((2, 1024, 8))
    ao, bo = rng.standard_normal((2, 8, 512)) / 22, 0.1 * rng.standard_normal((2, hid, 8))
    aq, bq, ao, bo = (v.astype(np.float32) for v in (aq, bq, ao, bo))
    ids = np.array([0, 1, -1, 1, 0, 0], np.int32)
    d = lambda v: to_dev(v, dev)  # noqa: E731
    qkv = lib.q8_linear_lora(d(wq), 1024, hid, d(x), d(aq), d(bq), d(ids), sections=parts)
    mid = qkv[:, :512] * 0.01
    out = lib.q8_linear_lora(d(wo), hid, 512, mid.contiguous(), d(ao), d(bo), d(ids))
    res = d(x) + 0.1 * out
    y = lib.q8_moe_layer(d(wr), d(gu), d(dn), e, f, hid, res, k)

    def lora(w, n, kk, v, a, b, cut):
        o = oracle.q8_linear_ref(w, n, kk, v)
        for t, i in enumerate(ids):
            if i >= 0:
                at = 0
                for p, rows in enumerate(cut):
                    o[t, at:at + rows] += b[i, at:at + rows].astype(np.float64) @ (
                        a[i, 8 * p:8 * p + 8].astype(np.float64) @ v[t])
                    at += rows
        return o

    r_qkv = lora(wq, 1024, hid, x.astype(np.float64), aq, bq, parts)
    r_out = lora(wo, hid, 512, 0.01 * r_qkv[:, :512], ao, bo, [hid])
    r_res = x + 0.1 * r_out
    idx, _ = lib.moe_route_topk(res, d(wr), k, True)
    idx = idx.cpu().numpy()
    p = np.take_along_axis(oracle.softmax_ref(oracle.router_logits_ref(r_res, wr)), idx.astype(np.int64), axis=1)
    ref = moe_mixture_grouped_ref(gu, dn, e, f, hid, r_res, idx, p / p.sum(axis=1, keepdims=True))
    assert_close(y.cpu().numpy(), ref, "decode step", tol=1e-4)
