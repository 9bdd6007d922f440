"""GPU parity of the adapter calls (q8_linear_lora, q8_linear_fused_gate_up_silu_lora,
lora_add, lora_gate_up_silu) against the definition in float64.

Error bounds (elementwise, from the inputs alone).  With u = 2^-24 and
gamma(d) = d u / (1 - d u), a float32 sum whose terms each pass through at most d roundings
is off by at most gamma(d) times the sum of the terms' magnitudes.  The shared product's
terms pass through a block's chain (32), a chain over at most k / 32 blocks and a tree of
at most 16 levels; an inner product of A through a chain of at most k / 8 (a matrix-core
chain of every eighth product is the longest form) and a tree, the outer one through at most
`rank` more.  The shared product may take x as a 32-bit fixed-point number of the row's
largest power of two, off by at most 2^-30 of the row's largest magnitude."""

from __future__ import annotations

import numpy as np
import pytest

import oracle
import workloads as wl
from gpu_util import say, to_dev, torch_dev

pytestmark = pytest.mark.gpu

TYPES = ("float32", "float16", "bfloat16")


def gamma(d):
    return d * 2.0 ** -24 / (1 - d * 2.0 ** -24)


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


class Case:
    """Seeded adapters beside a product of n outputs and width k, on host and device."""

    def __init__(self, env, seed, m, n, k, count, rank, kind, sections=None, ranks=True, none=0.2, scaled=True):
        _, torch, dev = env
        self.env, self.m, self.n, self.k, self.rank, self.count = env, m, n, k, rank, count
        self.sections = sections
        r = np.random.default_rng(seed)
        parts = sections or [n]
        dt = getattr(torch, kind)
        a = torch.from_numpy((r.standard_normal((count, len(parts) * rank, k)) / np.sqrt(k)).astype(np.float32))
        b = torch.from_numpy((0.3 * r.standard_normal((count, n, rank))).astype(np.float32))
        self.a, self.b = a.to(dt).to(dev), b.to(dt).to(dev)
        self.a64, self.b64 = a.to(dt).double().numpy(), b.to(dt).double().numpy()
        self.scale = r.uniform(-2, 2, count).astype(np.float32) if scaled else np.ones(count, np.float32)
        self.ranks = r.integers(0, rank + 1, count).astype(np.int32) if ranks else None
        self.adapter = np.where(r.random(m) < none, -1, r.integers(0, max(count, 1), m)).astype(np.int32)
        self.x = wl.activations(seed + 1, m, k)
        self.parts = parts
        self.args = (self.a, self.b, to_dev(self.adapter, dev))
        self.more = dict(scale=to_dev(self.scale, dev) if scaled else None,
                         ranks=to_dev(self.ranks, dev) if ranks else None, sections=sections)
        self.xd = to_dev(self.x, dev)

    def delta(self):
        """(D, its error bound), [m][n] float64."""
        d, bound = np.zeros((self.m, self.n)), np.zeros((self.m, self.n))
        x = self.x.astype(np.float64)
        for t, e in enumerate(self.adapter):
            if not 0 <= e < self.count:
                continue
            r = self.rank if self.ranks is None else int(self.ranks[e])
            at = 0
            for p, rows in enumerate(self.parts):
                a = self.a64[e, p * self.rank:p * self.rank + r]
                b = self.b64[e, at:at + rows, :r]
                d[t, at:at + rows] = self.scale[e] * (b @ (a @ x[t]))
                bound[t, at:at + rows] = abs(self.scale[e]) * (np.abs(b) @ (np.abs(a) @ np.abs(x[t])))
                at += rows
        return d, gamma(self.k / 8 + 16 + self.rank + 4) * bound


def packed(seed, n, k):
    w, q, d = wl.q8_weight(seed, n, k)
    return w, oracle.dequantize_q8_0(w, n, k)


def product(w64, x):
    """(x W^T, the error bound of a float32-accurate evaluation)."""
    x = x.astype(np.float64)
    k = x.shape[1]
    fixed = 2.0 ** -30 * np.abs(x).max(axis=1, initial=0)[:, None] * np.abs(w64).sum(axis=1)[None, :]
    return x @ w64.T, gamma(k / 32 + 52) * (np.abs(x) @ np.abs(w64).T) + fixed


def added(y, ye, d, de):
    """y + D and its bound: one more rounding of the sum, and of the correction before it."""
    s = y + d
    return s, ye + de + 2.0 ** -23 * (np.abs(y) + np.abs(d))


def activated(v, ve, f):
    """SiLU(g) u and its bound: |SiLU'| <= 1.1; the device's exp is off by at most
    (|g| + 1) 2^-23 relatively (the argument's two roundings, one ulp), the divide, product
    and sum around it by at most 6 more half ulps."""
    g, u, ge, ue = v[:, :f], v[:, f:], ve[:, :f], ve[:, f:]
    h = oracle.silu_ref(g) * u
    return h, 1.1 * ge * (np.abs(u) + ue) + np.abs(oracle.silu_ref(g)) * ue + (np.abs(g) + 8) * 2.0 ** -23 * np.abs(h)


def check(got, want, bound, what):
    got = got.cpu().numpy().astype(np.float64)
    off = np.abs(got - want)
    worst = float((off / np.maximum(bound, 1e-300)).max()) if off.size else 0.0
    say(f"{what}: worst error {worst:.3f} of its bound, rel {np.linalg.norm(off) / max(np.linalg.norm(want), 1e-300):.1e}")
    assert np.all(off <= bound), what


# m, n, k, adapters, rank, sections: one row to many, odd outputs, sections ending inside a tile,
# an empty section, one and many K slices, widths above what registers hold
LINEARS = [(1, 64, 256, 1, 8, None), (1, 2001, 1024, 3, 16, [1500, 501]), (2, 16, 256, 2, 8, None),
           (3, 1, 512, 2, 24, None), (4, 100, 1280, 4, 8, [7, 90, 3]), (5, 333, 2048, 5, 64, [0, 333]),
           (9, 48, 3840, 3, 16, [16, 16, 16]), (16, 6144, 4096, 8, 16, [4096, 1024, 1024]),
           (17, 130, 768, 17, 40, None), (33, 77, 4352, 2, 256, None), (64, 200, 1536, 6, 8, [50, 50, 50, 50]),
           (255, 129, 512, 30, 16, None), (3, 40, 12288, 2, 8, None), (6, 24, 16384, 2, 16, [8, 16]),
           (2, 18, 20480, 1, 8, None),
           # rows of 17 to 64 slices cut into ranges: uneven ones, more rows than one pass takes,
           # more tiles than blocks, many rows
           (1, 4096, 5888, 1, 8, None), (13, 700, 8192, 3, 8, [350, 350]), (64, 33, 8448, 4, 8, None),
           (65, 20, 4352, 4, 8, None), (7, 9000, 4352, 2, 8, None), (130, 90, 8192, 9, 16, [30, 60]),
           (255, 333, 5120, 3, 8, None)]


@pytest.mark.parametrize("m,n,k,count,rank,sections", LINEARS)
def test_linear(q8, m, n, k, count, rank, sections):
    lib, torch, dev = q8
    kind = TYPES[(m + n) % 3]
    say(f"q8_linear_lora m={m} n={n} k={k} adapters={count} rank={rank} {kind}")
    c = Case(q8, 100 * m + n, m, n, k, count, rank, kind, sections)
    w, w64 = packed(7 + n, n, k)
    y = lib.q8_linear_lora(to_dev(w, dev), n, k, c.xd, *c.args, **c.more)
    check(y, *added(*product(w64, c.x), *c.delta()), "q8_linear_lora")


@pytest.mark.parametrize("m,f,k,count,rank,split", [(1, 128, 256, 1, 16, True), (3, 33, 1024, 2, 8, True),
                                                    (8, 1000, 2048, 4, 32, True), (21, 40, 4096, 3, 8, False),
                                                    (70, 24, 768, 5, 16, True), (5, 7, 12288, 2, 8, False),
                                                    (255, 17, 512, 9, 24, True), (4, 19, 16640, 2, 8, True),
                                                    (18, 300, 5888, 3, 8, True)])
def test_gate_up(q8, m, f, k, count, rank, split):
    lib, torch, dev = q8
    kind = TYPES[(m + f) % 3]
    say(f"q8_linear_fused_gate_up_silu_lora m={m} f={f} k={k} adapters={count} rank={rank} {kind}")
    c = Case(q8, 100 * m + f, m, 2 * f, k, count, rank, kind, [f, f] if split else None)
    w, w64 = packed(8 + f, 2 * f, k)
    h = lib.q8_linear_fused_gate_up_silu_lora(to_dev(w, dev), f, k, c.xd, *c.args, **c.more)
    check(h, *activated(*added(*product(w64 * 1.0, c.x), *c.delta()), f), "q8_linear_fused_gate_up_silu_lora")


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k,count,rank,sections", [(1, 300, 256, 2, 8, None), (7, 65, 512, 3, 16, [1, 64]),
                                                       (64, 200, 768, 2, 24, [72, 128]), (65, 31, 1024, 7, 8, None),
                                                       (130, 515, 2048, 3, 64, [256, 259]),
                                                       (600, 257, 256, 40, 16, None), (300, 64, 512, 4, 256, None),
                                                       (1025, 96, 1280, 1, 8, [32, 32, 32])])
def test_add(q8, m, n, k, count, rank, sections, kind):
    lib, torch, dev = q8
    say(f"lora_add m={m} n={n} k={k} adapters={count} rank={rank} {kind}")
    c = Case(q8, 10 * m + n, m, n, k, count, rank, kind, sections)
    y = wl.activations(5 + m, m, n)
    out = lib.lora_add(to_dev(y, dev), c.xd, *c.args, **c.more)
    check(out, *added(y.astype(np.float64), 0, *c.delta()), "lora_add")


@pytest.mark.parametrize("m,f,k,count,rank,split", [(1, 64, 256, 1, 8, True), (6, 33, 512, 3, 16, False),
                                                    (90, 150, 1024, 4, 24, True), (300, 129, 512, 20, 32, True),
                                                    (700, 40, 256, 2, 64, True)])
def test_act(q8, m, f, k, count, rank, split):
    lib, torch, dev = q8
    kind = TYPES[m % 3]
    say(f"lora_gate_up_silu m={m} f={f} k={k} adapters={count} rank={rank} {kind}")
    c = Case(q8, 10 * m + f, m, 2 * f, k, count, rank, kind, [f, f] if split else None)
    gu = wl.activations(6 + m, m, 2 * f)
    h = lib.lora_gate_up_silu(to_dev(gu, dev), c.xd, *c.args, **c.more)
    check(h, *activated(*added(gu.astype(np.float64), 0, *c.delta()), f), "lora_gate_up_silu")


@pytest.mark.parametrize("m,gate_up", [(256, False), (300, True)])
def test_prefill_is_the_packed_product_and_the_correction(q8, m, gate_up):
    """From 256 rows on the shared product is q8_linear's own."""
    lib, torch, dev = q8
    n, k = 192, 1024
    c = Case(q8, 60, m, n, k, 5, 16, "bfloat16", [96, 96])
    w = to_dev(wl.q8_weight(61, n, k)[0], dev)
    base = lib.q8_linear(w, n, k, c.xd).cpu().numpy().astype(np.float64)
    if gate_up:
        h = lib.q8_linear_fused_gate_up_silu_lora(w, n // 2, k, c.xd, *c.args, **c.more)
        check(h, *activated(*added(base, 0, *c.delta()), n // 2), "prefill gate_up")
    else:
        y = lib.q8_linear_lora(w, n, k, c.xd, *c.args, **c.more)
        check(y, *added(base, 0, *c.delta()), "prefill linear")


def test_defaults_no_adapters_and_empty_calls(q8):
    """No scale, ranks or sections; rows without an adapter; a stack of none; no rows."""
    lib, torch, dev = q8
    n, k = 70, 512
    w, w64 = packed(20, n, k)
    wd = to_dev(w, dev)
    c = Case(q8, 21, 6, n, k, 2, 8, "float16", ranks=False, scaled=False, none=0.0)
    check(lib.q8_linear_lora(wd, n, k, c.xd, *c.args), *added(*product(w64, c.x), *c.delta()), "defaults")
    outside = torch.tensor([-1, 2, 2 ** 31 - 1, -2 ** 31, -7, 100], dtype=torch.int32, device=dev)
    check(lib.q8_linear_lora(wd, n, k, c.xd, c.a, c.b, outside), *product(w64, c.x), "ids outside the stack")
    none = lib.q8_linear_lora(wd, n, k, c.xd, c.a[:0], c.b[:0], outside)
    assert torch.equal(none, lib.q8_linear_lora(wd, n, k, c.xd, c.a, c.b, outside))
    y = torch.randn(6, n, device=dev)
    assert torch.equal(lib.lora_add(y, c.xd, c.a[:0], c.b[:0], outside), y)
    assert lib.q8_linear_lora(wd, n, k, c.xd[:0], c.a, c.b, outside[:0]).shape == (0, n)
    assert lib.lora_add(y[:0], c.xd[:0], c.a, c.b, outside[:0]).shape == (0, n)


@pytest.mark.parametrize("m", [2, 40, 300])
def test_unused_entries_may_hold_anything(q8, m):
    """Entries of A and B past an adapter's own rank, ranks below 0 and above `rank`, and the
    whole of an adapter that no row names."""
    lib, torch, dev = q8
    n, k, rank = 90, 512, 16
    c = Case(q8, 30 + m, m, n, k, 4, rank, "bfloat16", [45, 45], none=0.0)
    c.adapter[c.adapter == 3] = 0
    c.ranks[:] = [5, 0, rank, rank]
    a, b = c.a.clone(), c.b.clone()
    a.view(4, 2, rank, k)[0, :, 5:] = float("nan")
    b[0, :, 5:] = float("inf")
    a[1], b[1] = float("nan"), float("nan")
    a[3], b[3] = float("inf"), float("nan")
    args = (a, b, to_dev(c.adapter, dev))
    ranks = torch.tensor([5, -3, 1000, 8], dtype=torch.int32, device=dev)
    y = wl.activations(31, m, n)
    out = lib.lora_add(to_dev(y, dev), c.xd, *args, scale=c.more["scale"], ranks=ranks, sections=[45, 45])
    check(out, *added(y.astype(np.float64), 0, *c.delta()), "lora_add")
    w, w64 = packed(32, n, k)
    if m < 256:
        out = lib.q8_linear_lora(to_dev(w, dev), n, k, c.xd, *args, scale=c.more["scale"], ranks=ranks,
                                 sections=[45, 45])
        check(out, *added(*product(w64, c.x), *c.delta()), "q8_linear_lora")


def test_rows_that_are_not_finite_stay_apart(q8):
    lib, torch, dev = q8
    n, k, m = 50, 768, 9
    c = Case(q8, 40, m, n, k, 2, 8, "float32", [25, 25])
    w, w64 = packed(41, n, k)
    wd = to_dev(w, dev)
    good = lib.q8_linear_lora(wd, n, k, c.xd, *c.args, **c.more)
    x = c.xd.clone()
    x[2, 5], x[4, 700], x[8, 0] = float("nan"), float("inf"), float("-inf")
    for y in (lib.q8_linear_lora(wd, n, k, x, *c.args, **c.more),
              lib.q8_linear_fused_gate_up_silu_lora(wd, n // 2, k, x, *c.args, **c.more)):
        assert not torch.isfinite(y[[2, 4, 8]]).any()
        assert torch.isfinite(y[[0, 1, 3, 5, 6, 7]]).all()
    y = lib.q8_linear_lora(wd, n, k, x, *c.args, **c.more)
    assert torch.equal(y[[0, 1, 3, 5, 6, 7]], good[[0, 1, 3, 5, 6, 7]])


@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -60, 2.0 ** 60, 0.0])
def test_rows_of_any_magnitude(q8, scale):
    """The same rows times a power of two give the same outputs times it (down to where
    products leave the normal float32 range), zero rows give zeros."""
    lib, torch, dev = q8
    n, k, m = 40, 512, 5
    c = Case(q8, 50, m, n, k, 2, 8, "float32")
    w, w64 = packed(51, n, k)
    x = (c.x * scale).astype(np.float32)
    y = lib.q8_linear_lora(to_dev(w, dev), n, k, to_dev(x, dev), *c.args, **c.more).cpu().numpy()
    c.x = x
    want, bound = added(*product(w64, x), *c.delta())
    assert np.all(np.abs(y - want) <= bound + 2.0 ** -126), scale


@pytest.mark.parametrize("n,k,most", [(200, 1024, 255), (96, 4096, 255), (300, 768, 100), (70, 5888, 64),
                                      (33, 16384, 64)])
def test_a_row_depends_on_itself_alone(q8, n, k, most):
    """Any subset of two rows and more gives the same bits, one row twice included."""
    lib, torch, dev = q8
    c = Case(q8, 75 + n, most, n, k, 5, 16, "bfloat16", [n // 2, n - n // 2])
    w = to_dev(wl.q8_weight(76, n, k)[0], dev)
    a, b, ids = c.args
    whole = lib.q8_linear_lora(w, n, k, c.xd, a, b, ids, **c.more)
    rng = np.random.default_rng(77)
    for m in (1, 2, 4, 5, 8, 9, 13, 17, 40):
        rows = torch.from_numpy(np.sort(rng.choice(most, m, replace=False))).to(dev)
        if m == 1:
            rows = rows.repeat(2)
        part = lib.q8_linear_lora(w, n, k, c.xd[rows].contiguous(), a, b, ids[rows].contiguous(), **c.more)
        assert torch.equal(part, whole[rows]), m
    for _ in range(5):
        assert torch.equal(lib.q8_linear_lora(w, n, k, c.xd, a, b, ids, **c.more), whole)


@pytest.mark.parametrize("m", [20, 300])
def test_adding_does_not_depend_on_the_other_rows(q8, m):
    """Within a form (few rows, many rows) a row's bits are its own."""
    lib, torch, dev = q8
    n, k = 150, 512
    c = Case(q8, 78 + m, m, n, k, 6, 24, "float16", [70, 80], none=0.3)
    a, b, ids = c.args
    y = torch.randn(m, n, device=dev)
    whole = lib.lora_add(y, c.xd, a, b, ids, **c.more)
    turned = torch.randperm(m, device=dev)
    part = lib.lora_add(y[turned], c.xd[turned], a, b, ids[turned], **c.more)
    assert torch.equal(part, whole[turned])
    assert torch.equal(whole[ids < 0], y[ids < 0])


@pytest.mark.parametrize("n,k,rank,sections", [(6144, 4096, 16, [4096, 1024, 1024]), (517, 8192, 40, None),
                                               (4099, 8192, 8, [4000, 99]), (3000, 12288, 64, None),
                                               (901, 16384, 24, [900, 1]), (24, 20480, 8, None)])
def test_one_row(q8, n, k, rank, sections):
    """The correction behind the one-row kernel, in all its forms; beyond it; and without a
    correction the same values as the linears alone."""
    lib, torch, dev = q8
    f = n // 2
    c = Case(q8, 65 + n, 1, n, k, 3, rank, TYPES[n % 3], sections, none=0.0)
    w, w64 = packed(66, n, k)
    wd = to_dev(w, dev)
    y, bound = added(*product(w64, c.x), *c.delta())
    got = lib.q8_linear_lora(wd, n, k, c.xd, *c.args, **c.more)
    check(got, y, bound, "q8_linear_lora")
    if n % 2 == 0:
        h = lib.q8_linear_fused_gate_up_silu_lora(wd, f, k, c.xd, *c.args, **c.more)
        check(h, *activated(y, bound, f), "q8_linear_fused_gate_up_silu_lora")
    for a, b, i in ((c.a[:0], c.b[:0], 0), (c.a, c.b, -1), (c.a, c.b, 3)):
        ids = torch.tensor([i], dtype=torch.int32, device=dev)
        more = dict(sections=sections)
        assert torch.equal(lib.q8_linear_lora(wd, n, k, c.xd, a, b, ids, **more), lib.q8_linear(wd, n, k, c.xd))
        if n % 2 == 0:
            assert torch.equal(lib.q8_linear_fused_gate_up_silu_lora(wd, f, k, c.xd, a, b, ids, **more),
                               lib.q8_linear_fused_gate_up_silu(wd, f, k, c.xd))
    x = c.xd.clone()
    x[0, k - 1] = float("inf")
    assert not torch.isfinite(lib.q8_linear_lora(wd, n, k, x, *c.args, **c.more)).any()


# The matrix-core form: calls whose rows would read 160 MB of their adapters.  Few rows of wide
# and many of narrow adapters, odd outputs, sections that end inside a block of 128 outputs,
# adapters with fewer rows than a tile, one adapter for all, one part of k and several
MANY = [(48, 129, 8192, 2, 256, None), (64, 33, 16384, 3, 256, [33]), (420, 77, 1280, 7, 96, [30, 47]),
        (700, 515, 512, 40, 64, [256, 3, 256]), (1300, 57, 256, 256, 256, None), (5200, 1301, 768, 1, 8, [1, 1300]),
        (2111, 640, 1024, 5, 24, [160, 160, 160, 160])]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("m,n,k,count,rank,sections", MANY)
def test_add_many_rows(q8, m, n, k, count, rank, sections, kind):
    lib, torch, dev = q8
    say(f"lora_add m={m} n={n} k={k} adapters={count} rank={rank} {kind}")
    c = Case(q8, 11 * m + n, m, n, k, count, rank, kind, sections)
    y = wl.activations(5 + m, m, n)
    yd = to_dev(y, dev)
    check(lib.lora_add(yd, c.xd, *c.args, **c.more), *added(y.astype(np.float64), 0, *c.delta()), "lora_add")


@pytest.mark.parametrize("m,f,k,count,rank,split", [(420, 77, 1280, 7, 96, True), (1100, 301, 512, 30, 64, True),
                                                    (900, 150, 2048, 3, 40, False), (48, 65, 8192, 2, 256, True)])
def test_act_many_rows(q8, m, f, k, count, rank, split):
    lib, torch, dev = q8
    kind = TYPES[m % 3]
    say(f"lora_gate_up_silu m={m} f={f} k={k} adapters={count} rank={rank} {kind}")
    c = Case(q8, 11 * m + f, m, 2 * f, k, count, rank, kind, [f, f] if split else [f + 5, f - 5])
    gu = wl.activations(6 + m, m, 2 * f)
    h = lib.lora_gate_up_silu(to_dev(gu, dev), c.xd, *c.args, **c.more)
    check(h, *activated(*added(gu.astype(np.float64), 0, *c.delta()), f), "lora_gate_up_silu")


def test_many_rows_use_what_is_theirs(q8):
    """In the matrix-core form: entries past a rank and adapters nobody names may hold
    anything, rows that are not finite stay apart, a row's bits are its own, in place or
    not, in a graph or not."""
    lib, torch, dev = q8
    m, n, k, rank = 800, 300, 1024, 64
    c = Case(q8, 63, m, n, k, 4, rank, "bfloat16", [140, 160])
    c.adapter[c.adapter == 3] = 0
    c.ranks[:] = [5, 0, rank, rank]
    a, b = c.a.clone(), c.b.clone()
    a.view(4, 2, rank, k)[0, :, 5:] = float("nan")
    b[0, :, 5:] = float("inf")
    a[1], b[1] = float("nan"), float("nan")
    a[3], b[3] = float("inf"), float("nan")
    ids = to_dev(c.adapter, dev)
    more = dict(scale=c.more["scale"], ranks=torch.tensor([5, -3, 1000, 8], dtype=torch.int32, device=dev),
                sections=c.sections)
    y = wl.activations(64, m, n)
    yd = to_dev(y, dev)
    got = lib.lora_add(yd, c.xd, a, b, ids, **more)
    check(got, *added(y.astype(np.float64), 0, *c.delta()), "lora_add")
    assert torch.equal(got[ids < 0], yd[ids < 0])
    turned = torch.randperm(m, device=dev)
    assert torch.equal(lib.lora_add(yd[turned], c.xd[turned], a, b, ids[turned], **more), got[turned])
    x = c.xd.clone()
    bad = torch.nonzero(ids == 2).flatten()[:3]
    x[bad[0], 5], x[bad[1], 700], x[bad[2], 0] = float("nan"), float("inf"), float("-inf")
    out = lib.lora_add(yd, x, a, b, ids, **more)
    rest = torch.ones(m, dtype=torch.bool, device=dev)
    rest[bad] = False
    assert not torch.isfinite(out[bad]).any() and torch.equal(out[rest], got[rest])
    ws = torch.empty(lib.lora_workspace_bytes(m, rank, 2), dtype=torch.uint8, device=dev)
    z = yd.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.lora_add(z, c.xd, a, b, ids, **more, out=z, workspace=ws)
    for _ in range(3):
        z.copy_(yd)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, got)


def test_more_outputs_and_adapters_than_a_grid_holds(q8):
    """Row tiles of 256 adapters times 2^23 outputs pass 2^32 threads: the other form."""
    lib, torch, dev = q8
    m, n, k, rank, count = 300, 1 << 23, 256, 8, 256
    a = torch.ones((count, rank, k), dtype=torch.bfloat16, device=dev)
    b = torch.zeros((count, n, rank), dtype=torch.bfloat16, device=dev)
    b[3, -5:] = 0.25
    x = torch.ones((m, k), device=dev)
    ids = (torch.arange(m, device=dev) % count).int()
    y = torch.zeros((m, n), device=dev)
    assert lib.lora_add(y, x, a, b, ids, out=y) is y
    want = torch.where(ids == 3, rank * k * 0.25, 0.0)
    assert torch.equal(y[:, -5:], want[:, None].expand(m, 5)) and not y[:, :-5].any()


def test_strided_rows_and_rows_behind_the_last(q8):
    """Padded leading dimensions; what lies outside the outputs stays as it was."""
    lib, torch, dev = q8
    m, n, k = 5, 67, 512
    c = Case(q8, 70, m, n, k, 3, 16, "float16", [30, 37])
    w, w64 = packed(71, n, k)
    wd = to_dev(w, dev)
    x = torch.full((m + 2, k + 8), float("nan"), device=dev)
    x[:m, :k] = c.xd
    buf = torch.full((m + 3, n + 5), 7.0, device=dev)
    out = lib.q8_linear_lora(wd, n, k, x[:m, :k], *c.args, **c.more, out=buf[1:m + 1, :n])
    assert torch.equal(out, lib.q8_linear_lora(wd, n, k, c.xd, *c.args, **c.more))
    y = torch.randn(m, n, device=dev)
    ypad = torch.full((m, n + 3), float("nan"), device=dev)
    ypad[:, :n] = y
    buf2 = torch.full((m + 3, n + 5), 7.0, device=dev)
    got = lib.lora_add(ypad[:, :n], x[:m, :k], *c.args, **c.more, out=buf2[1:m + 1, :n])
    assert torch.equal(got, lib.lora_add(y, c.xd, *c.args, **c.more))
    for b in (buf, buf2):
        assert (b[0] == 7).all() and (b[m + 1:] == 7).all() and (b[1:m + 1, n:] == 7).all()
    inplace = y.clone()
    assert torch.equal(lib.lora_add(inplace, c.xd, *c.args, **c.more, out=inplace), got)


@pytest.mark.parametrize("m", [3, 300])
def test_beside_every_format_and_the_integer_path(q8, m):
    """lora_add and lora_gate_up_silu beside the products of the other packed formats."""
    lib, torch, dev = q8
    f, k = 32, 512
    c = Case(q8, 80, m, 2 * f, k, 3, 8, "bfloat16", [f, f])
    makers = {"q4_0": wl.q4_0_weight, "q4_k": wl.q4_k_weight, "q5_k": wl.q5_k_weight, "q6_k": wl.q6_k_weight}
    for name, make in makers.items():
        w = to_dev(make(81, 2 * f, k)[0], dev)
        gu = getattr(lib, f"{name}_linear")(w, 2 * f, k, c.xd)
        base = gu.cpu().numpy().astype(np.float64)
        check(lib.lora_add(gu, c.xd, *c.args, **c.more), *added(base, 0, *c.delta()), f"{name} + lora_add")
        check(lib.lora_gate_up_silu(gu, c.xd, *c.args, **c.more), *activated(*added(base, 0, *c.delta()), f),
              f"{name} + lora_gate_up_silu")
    w = to_dev(wl.q8_weight(82, 2 * f, k)[0], dev)
    y = lib.q8_linear_q8act(w, 2 * f, k, *lib.q8_quantize_act(c.xd))
    check(lib.lora_add(y, c.xd, *c.args, **c.more), *added(y.cpu().numpy().astype(np.float64), 0, *c.delta()),
          "q8act + lora_add")


def test_offsets_past_32_bits(q8):
    """The last adapter of a stack of more than 2^32 elements; outputs past 2^32 elements."""
    lib, torch, dev = q8
    count, rank, k, n, m = 256, 256, 16640, 64, 2
    a = torch.zeros((count, 4 * rank, k), dtype=torch.bfloat16, device=dev)
    b = torch.zeros((count, n, rank), dtype=torch.bfloat16, device=dev)
    assert a.numel() > 2 ** 32
    a[-1, 3 * rank:, :] = 2.0 ** -7
    b[-1, 48:, :] = 0.5
    x = torch.ones((m, k), device=dev)
    adapter = torch.tensor([count - 1, 0], dtype=torch.int32, device=dev)
    y = lib.lora_add(torch.zeros((m, n), device=dev), x, a, b, adapter, sections=[16, 16, 16, 16])
    want = torch.zeros((m, n), device=dev)
    want[0, 48:] = 256 * 0.5 * (k * 2.0 ** -7)   # exact in float32
    assert torch.equal(y, want)
    del a
    rows, ld, n = 300, 1 << 24, 40
    c = Case(q8, 91, rows, n, 256, 2, 8, "float32")
    big = torch.zeros(rows * ld, device=dev).view(rows, ld)
    assert (rows - 1) * ld > 2 ** 32
    got = lib.lora_add(big[:, :n], c.xd, *c.args, **c.more, out=big[:, 64:64 + n])
    assert torch.equal(got.contiguous(), lib.lora_add(torch.zeros((rows, n), device=dev), c.xd, *c.args, **c.more))


def test_streams_workspaces_and_graphs(q8):
    """Two streams at once with workspaces of their own; a captured call replayed between
    eager work; a reused workspace's old contents do not matter."""
    lib, torch, dev = q8
    m, n, k = 12, 512, 2048
    c = Case(q8, 95, m, n, k, 4, 16, "bfloat16", [256, 256])
    w = to_dev(wl.q8_weight(96, n, k)[0], dev)
    size = lib.q8_linear_lora_workspace_bytes(m, n, k, 16, 2)
    ws = [torch.full((size,), 0xFF, dtype=torch.uint8, device=dev) for _ in range(3)]
    want = lib.q8_linear_lora(w, n, k, c.xd, *c.args, **c.more)
    want_h = lib.q8_linear_fused_gate_up_silu_lora(w, n // 2, k, c.xd, *c.args, **c.more)
    outs = [torch.empty((m, n), device=dev), torch.empty((m, n // 2), device=dev)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s[0]):
            lib.q8_linear_lora(w, n, k, c.xd, *c.args, **c.more, out=outs[0], workspace=ws[0])
        with torch.cuda.stream(s[1]):
            lib.q8_linear_fused_gate_up_silu_lora(w, n // 2, k, c.xd, *c.args, **c.more, out=outs[1], workspace=ws[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want_h)
    x = c.xd.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lib.q8_linear_lora(w, n, k, x, *c.args, **c.more, workspace=ws[2])
        z = lib.lora_add(y, x, *c.args, **c.more)
    for i in range(4):
        x.copy_(c.xd * (i + 1))
        ws[2].fill_(i)
        g.replay()
        torch.cuda.synchronize()
        eager = lib.q8_linear_lora(w, n, k, x, *c.args, **c.more)
        assert torch.equal(y, eager) and torch.equal(z, lib.lora_add(eager, x, *c.args, **c.more)), i


def test_binding_refusals(q8):
    lib, torch, dev = q8
    m, n, k = 3, 64, 512
    c = Case(q8, 98, m, n, k, 2, 8, "float16")
    w = to_dev(wl.q8_weight(99, n, k)[0], dev)
    a, b, ad = c.args
    y = torch.zeros((m, n), device=dev)

    def bad(*args, err=ValueError, fn=None, **kw):
        with pytest.raises(err):
            (fn or (lambda *p, **q: lib.q8_linear_lora(w, n, k, c.xd, *p, **q)))(*args, **kw)

    bad(a, b.float(), ad)
    bad(a.double(), b.double(), ad)
    bad(a[:1], b, ad)
    bad(a, b[:, :10], ad)
    bad(a, b.transpose(1, 2), ad)
    bad(a, b, ad.long())
    bad(a, b, ad[:2])
    bad(a, b, ad.cpu())
    bad(a, b, ad, scale=torch.ones(3, device=dev))
    bad(a, b, ad, ranks=torch.ones(2, device=dev))
    bad(a, b, ad, sections=[60, 3])
    bad(a, b, ad, sections=[32, 32])          # a holds one section's rows
    bad(a, b, ad, out=torch.empty((m, n + 1), device=dev))
    bad(a, b, ad, err=lib.Q8Error, workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    bad(a[:, :4].contiguous(), b[:, :, :4].contiguous(), ad, err=lib.Q8Error)   # rank 4
    bad(y.double(), c.xd, a, b, ad, fn=lib.lora_add)
    bad(y[:, :63], c.xd, a, b, ad, fn=lib.lora_add)
    bad(y[:2], c.xd, a, b, ad, fn=lib.lora_add)
    bad(torch.zeros((m, 63), device=dev), c.xd, a, b, ad, fn=lib.lora_gate_up_silu)
