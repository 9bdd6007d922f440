"""Argument errors of the adapter calls and the whole MoE layer at the C entry points, on the
host (no GPU needed): nothing below reaches a kernel."""

from __future__ import annotations

import ctypes
import threading

import pytest

q8 = pytest.importorskip("block_quantized_weight_linear_amd")
lib = q8.lib
from block_quantized_weight_linear_amd._binding import _Lora  # noqa: E402

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_DEVICE = range(6)
FAKE = 0x10000  # 256-byte aligned, never dereferenced
BIG = 1 << 40


def lora(n=64, a=FAKE, b=FAKE, ranks=None, scale=None, adapter=FAKE, sections=None, type=2, count=3, rank=16, ns=None):
    rows = (n,) if sections is None else sections
    return _Lora(a, b, ranks, scale, adapter, rows, type, count, rank, len(rows) if ns is None else ns)


def linear(lo=None, w=FAKE, n=64, k=256, x=FAKE, m=2, ldx=256, y=FAKE, ldy=64, ws=FAKE, size=BIG, fused=False, **kw):
    lo = lora(2 * n if fused else n, **kw) if lo is None else lo
    fn = lib.q8_linear_fused_gate_up_silu_lora if fused else lib.q8_linear_lora
    return fn(w, n, k, x, m, ldx, lo if lo != 0 else None, y, ldy, ws, size, None)


def beside(lo=None, y=FAKE, n=64, ldy=128, x=FAKE, m=2, k=256, ldx=256, out=FAKE, ldo=64, ws=FAKE, size=BIG,
           fused=False, **kw):
    lo = lora(2 * n if fused else n, **kw) if lo is None else lo
    fn = lib.lora_gate_up_silu if fused else lib.lora_add
    return fn(y, n, ldy, x, m, k, ldx, lo if lo != 0 else None, out, ldo, ws, size, None)


@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("call", [linear, beside])
def test_adapter_arguments(call, fused):
    def c(**kw):
        return call(fused=fused, **kw)

    n = 128 if fused else 64
    assert c(lo=0) == ERR_NULL
    assert c(type=3) == ERR_SHAPE and c(type=-1) == ERR_SHAPE
    assert c(count=-1) == ERR_SHAPE and c(count=257) == ERR_SHAPE
    for rank in (0, -8, 4, 12, 264, 1 << 30):
        assert c(rank=rank) == ERR_SHAPE, rank
    assert c(ns=0) == ERR_SHAPE and c(ns=5) == ERR_SHAPE
    assert c(sections=(n - 1,)) == ERR_SHAPE
    assert c(sections=(n, 1)) == ERR_SHAPE
    assert c(sections=(n + 8, -8)) == ERR_SHAPE
    assert c(sections=((1 << 62), (1 << 62), (1 << 62), n)) == ERR_SHAPE
    assert c(a=None) == ERR_NULL and c(b=None) == ERR_NULL and c(adapter=None) == ERR_NULL
    assert c(a=FAKE + 8) == ERR_ALIGN and c(b=FAKE + 2) == ERR_ALIGN
    assert c(ranks=FAKE + 1) == ERR_ALIGN and c(scale=FAKE + 2) == ERR_ALIGN and c(adapter=FAKE + 3) == ERR_ALIGN
    assert b"lora" in lib.q8_last_error()
    assert c(ws=None) == ERR_WORKSPACE and c(size=16) == ERR_WORKSPACE and c(ws=FAKE + 16) == ERR_ALIGN
    assert c(x=None) == ERR_NULL and c(x=FAKE + 4) == ERR_ALIGN and c(ldx=258) == ERR_ALIGN
    assert c(ldx=252) == ERR_SHAPE and c(k=128) == ERR_SHAPE and c(m=-1) == ERR_SHAPE and c(n=-1) == ERR_SHAPE
    assert c(m=(1 << 22) + 1) == ERR_SHAPE
    assert c(n=1 << 31) == ERR_SHAPE and c(n=(1 << 62)) == ERR_SHAPE and c(n=-(1 << 62)) == ERR_SHAPE
    # nothing to do: pointers may be anything
    assert c(m=0, a=None, b=None, adapter=None, x=None, y=None, ws=None) == OK
    assert c(n=0, sections=(0,), x=None, y=None, ws=None) == OK


def test_product_arguments():
    assert linear(w=None) == ERR_NULL and linear(y=None) == ERR_NULL and linear(w=FAKE + 8) == ERR_ALIGN
    assert linear(ldy=63) == ERR_SHAPE and linear(y=FAKE + 2) == ERR_ALIGN
    assert beside(y=None) == ERR_NULL and beside(out=None) == ERR_NULL
    assert beside(ldy=63) == ERR_SHAPE and beside(ldo=63) == ERR_SHAPE
    assert beside(ldy=127, fused=True) == ERR_SHAPE
    assert beside(y=FAKE + 2) == ERR_ALIGN and beside(out=FAKE + 1) == ERR_ALIGN
    assert beside(ldo=1 << 31) == ERR_SHAPE and beside(ldy=1 << 32) == ERR_SHAPE


def test_adapter_workspace_sizes():
    assert q8.lora_workspace_bytes(16, 16, 3) >= 16 * 48 * 4
    assert q8.lora_workspace_bytes(16, 12, 3) == 0 and q8.lora_workspace_bytes(-1, 16, 3) == 0
    assert q8.lora_workspace_bytes(16, 16, 5) == 0 and q8.lora_workspace_bytes(1 << 23, 16) == 0
    assert q8.q8_linear_lora_workspace_bytes(16, 64, 100, 16) == 0
    assert q8.q8_linear_lora_workspace_bytes(16, -1, 256, 16) == 0
    assert q8.q8_linear_lora_workspace_bytes(16, 64, 256, 264) == 0
    assert q8.q8_linear_lora_workspace_bytes(300, 128, 256, 16, 2) % 256 == 0
    assert lib.lora_workspace_bytes(4, None) == 0 and lib.q8_linear_lora_workspace_bytes(4, 4, 256, None) == 0
    need = q8.q8_linear_lora_workspace_bytes(2, 64, 256, 16)
    assert linear(size=need - 1) == ERR_WORKSPACE
    assert str(need).encode() in lib.q8_last_error()


def moe(wr=FAKE, gu=FAKE, dn=FAKE, e=8, f=256, h=256, x=FAKE, m=2, ldx=256, k=2, top_p=1.0, y=FAKE, ldy=256, ws=FAKE,
        size=BIG):
    return lib.q8_moe_layer(wr, gu, dn, e, f, h, x, m, ldx, k, 1, ctypes.c_float(top_p), y, ldy, ws, size, None)


def test_moe_layer_arguments():
    assert moe(h=100) == ERR_SHAPE and moe(f=0) == ERR_SHAPE and moe(h=16640, ldx=16640, ldy=16640) == ERR_SHAPE
    assert moe(e=0) == ERR_SHAPE and moe(e=257) == ERR_SHAPE
    assert moe(k=0) == ERR_SHAPE and moe(k=9) == ERR_SHAPE and moe(m=-1) == ERR_SHAPE
    assert moe(ldx=252) == ERR_SHAPE and moe(ldy=255) == ERR_SHAPE and moe(ldx=258) == ERR_ALIGN
    assert moe(m=1 << 24) == ERR_SHAPE
    for p in (0.0, -1.0, 1.01, float("nan"), float("inf")):
        assert moe(top_p=p) == ERR_SHAPE, p
    for name in ("wr", "gu", "dn", "x", "y"):
        assert moe(**{name: None}) == ERR_NULL, name
    for name in ("wr", "gu", "dn", "x"):
        assert moe(**{name: FAKE + 8}) == ERR_ALIGN, name
    assert moe(y=FAKE + 2) == ERR_ALIGN
    assert moe(ws=None) == ERR_WORKSPACE and moe(size=8) == ERR_WORKSPACE and moe(ws=FAKE + 16) == ERR_ALIGN
    assert b"q8_moe_layer" in lib.q8_last_error()
    assert moe(m=0, wr=None, gu=None, dn=None, x=None, y=None, ws=None) == OK
    need = q8.q8_moe_layer_workspace_bytes(2, 2, 8, 256, 256)
    assert need % 256 == 0 and moe(size=need - 1) == ERR_WORKSPACE
    for bad in ((2, 9, 8, 256, 256), (2, 2, 8, 100, 256), (-1, 2, 8, 256, 256), (2, 2, 0, 256, 256),
                (1 << 24, 2, 8, 256, 256)):
        assert q8.q8_moe_layer_workspace_bytes(*bad) == 0, bad


def test_error_text_stays_with_its_thread():
    assert moe(k=9) == ERR_SHAPE
    seen = []
    t = threading.Thread(target=lambda: seen.append((linear(rank=4), lib.q8_last_error())))
    t.start()
    t.join()
    assert seen[0][0] == ERR_SHAPE and b"rank=4" in seen[0][1]
    assert b"k=9" in lib.q8_last_error()
