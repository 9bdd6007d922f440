"""Argument errors of the 8-bit floating-point calls at the C entry points, on the host (no GPU
needed): nothing below reaches a kernel."""

from __future__ import annotations

import threading

import pytest

q8 = pytest.importorskip("block_quantized_weight_linear_amd")
lib = q8.lib

OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_WORKSPACE, ERR_DEVICE = range(6)
FAKE = 0x10000  # 256-byte aligned, never dereferenced
BIG = 1 << 50


def quantize(fn, x=FAKE, type=0, m=2, k=256, ld=None, pow2=0, q=FAKE, d=FAKE):
    return fn(x, type, m, k, k if ld is None else ld, pow2, q, d, None)


@pytest.mark.parametrize("fn", [lib.f8_quantize_act, lib.f8_quantize_weight])
def test_quantizers(fn):
    def c(**kw):
        return quantize(fn, **kw)

    for type in (-1, 3, 99):
        assert c(type=type) == ERR_SHAPE, type
    for k in (0, -16, 8, 24, 129, (1 << 20) + 16, 1 << 62):
        assert c(k=k, ld=max(k, 1)) == ERR_SHAPE, k
    most = 1 << (24 if fn is lib.f8_quantize_act else 20)
    assert c(m=-1) == ERR_SHAPE and c(m=most + 1) == ERR_SHAPE and c(m=1 << 62) == ERR_SHAPE
    assert c(m=most, k=1 << 20) == ERR_SHAPE  # their product
    assert c(ld=252) == ERR_SHAPE and c(ld=(1 << 30) + 4) == ERR_SHAPE
    assert c(ld=258) == ERR_ALIGN and c(ld=260, type=1) == ERR_ALIGN and c(ld=260, type=2) == ERR_ALIGN
    assert c(x=None) == ERR_NULL and c(q=None) == ERR_NULL and c(d=None) == ERR_NULL
    assert c(x=FAKE + 8) == ERR_ALIGN and c(q=FAKE + 8) == ERR_ALIGN and c(d=FAKE + 2) == ERR_ALIGN
    assert c(m=0, x=None, q=None, d=None) == OK


def linear(wq=FAKE, wd=FAKE, n=64, k=256, xq=FAKE, xd=FAKE, m=2, y=FAKE, type=2, ldy=None, gu=None, ldgu=0, fused=False):
    ldy = n if ldy is None else ldy
    if fused:
        return lib.f8_linear_fused_gate_up_silu(wq, wd, n, k, xq, xd, m, y, type, ldy, gu, ldgu, None)
    return lib.f8_linear(wq, wd, n, k, xq, xd, m, y, type, ldy, None)


@pytest.mark.parametrize("fused", [False, True])
def test_products(fused):
    def c(**kw):
        return linear(fused=fused, **kw)

    for type in (-1, 3):
        assert c(type=type) == ERR_SHAPE
    for k in (0, -16, 24, (1 << 20) + 16):
        assert c(k=k) == ERR_SHAPE, k
    top = 1 << (19 if fused else 20)
    for n in (-1, top + 1, 1 << 61, -(1 << 62)):
        assert c(n=n, ldy=1 << 30) == ERR_SHAPE, n
    assert c(m=-1) == ERR_SHAPE and c(m=(1 << 24) + 1) == ERR_SHAPE
    assert c(m=1 << 24, n=1 << 14) == ERR_SHAPE and c(m=1 << 24, k=1 << 14) == ERR_SHAPE and c(n=top, k=1 << 18) == ERR_SHAPE
    assert c(ldy=63) == ERR_SHAPE and c(ldy=(1 << 30) + 1) == ERR_SHAPE
    for name in ("wq", "wd", "xq", "xd", "y"):
        assert c(**{name: None}) == ERR_NULL, name
    for name, shift in (("wq", 8), ("xq", 8), ("wd", 2), ("xd", 1), ("y", 1)):
        assert c(**{name: FAKE + shift}) == ERR_ALIGN, name
    assert c(y=FAKE + 2, type=0) == ERR_ALIGN
    assert c(m=0, wq=None, wd=None, xq=None, xd=None, y=None) == OK
    assert c(n=0, wq=None, wd=None, xq=None, xd=None, y=None) == OK
    assert b"" == lib.q8_last_error()


def test_kept_products():
    assert linear(fused=True, gu=FAKE, ldgu=127) == ERR_SHAPE
    assert linear(fused=True, gu=FAKE + 1, ldgu=128) == ERR_ALIGN
    assert b"gu" in lib.q8_last_error()


def backward(wq=FAKE, wd=FAKE, n=64, k=256, xq=FAKE, xd=FAKE, m=2, gu=FAKE, ldgu=None, d=FAKE, type=2, ldd=None, dx=FAKE,
             lddx=None, dw=FAKE, lddw=None, ws=FAKE, size=BIG, fused=False):
    ldd, lddx, lddw = (n if ldd is None else ldd), (k if lddx is None else lddx), (k if lddw is None else lddw)
    if fused:
        return lib.f8_linear_fused_gate_up_silu_backward(wq, wd, n, k, xq, xd, m, gu, 2 * n if ldgu is None else ldgu, d,
                                                         type, ldd, dx, lddx, dw, lddw, ws, size, None)
    return lib.f8_linear_backward(wq, wd, n, k, xq, xd, m, d, type, ldd, dx, lddx, dw, lddw, ws, size, None)


@pytest.mark.parametrize("fused", [False, True])
def test_backward(fused):
    def c(**kw):
        return backward(fused=fused, **kw)

    assert c(type=3) == ERR_SHAPE and c(type=-1) == ERR_SHAPE
    assert c(k=24) == ERR_SHAPE and c(n=-1, ldd=1) == ERR_SHAPE and c(m=-1) == ERR_SHAPE and c(m=1 << 25) == ERR_SHAPE
    assert c(ldd=63) == ERR_SHAPE and c(lddx=255) == ERR_SHAPE and c(lddw=255) == ERR_SHAPE
    for name in ("wq", "wd", "xq", "xd", "d"):
        assert c(**{name: None}) == ERR_NULL, name
    for name, shift in (("wq", 8), ("xq", 8), ("wd", 2), ("xd", 1), ("d", 1), ("dx", 1), ("dw", 1)):
        assert c(**{name: FAKE + shift}) == ERR_ALIGN, name
    if fused:
        assert c(gu=None) == ERR_NULL and c(gu=FAKE + 1) == ERR_ALIGN and c(ldgu=127) == ERR_SHAPE
    # operands of a gradient that is not asked for
    assert c(dx=None, dw=None, wq=None, xq=None, d=None, ws=None) == OK
    assert c(dx=None, xq=None) == ERR_NULL and c(dw=None, wq=None) == ERR_NULL
    assert c(ws=None) == ERR_WORKSPACE and c(size=8) == ERR_WORKSPACE and c(ws=FAKE + 16) == ERR_ALIGN
    sizes = lib.f8_linear_fused_gate_up_silu_backward_workspace_bytes if fused else lib.f8_linear_backward_workspace_bytes
    for type in (0, 1, 2):
        need = sizes(2, 64, 256, type)
        assert need % 256 == 0 and need > 0
        assert c(type=type, size=need - 1) == ERR_WORKSPACE
        assert str(need).encode() in lib.q8_last_error()
    for bad in ((-1, 64, 256, 2), (2, -1, 256, 2), (2, 64, 24, 2), (2, 64, 256, 3), (1 << 25, 64, 256, 2),
                (2, 1 << 21, 256, 2), (1 << 24, 1 << 20, 256, 2), (2, 1 << 62, 256, 2)):
        assert sizes(*bad) == 0, bad
    # nothing to add up, nothing asked for: no pointer is looked at
    assert c(m=0, n=0, dx=None, dw=None) == OK


def test_error_text_stays_with_its_thread():
    assert linear(k=24) == ERR_SHAPE
    seen = []
    t = threading.Thread(target=lambda: seen.append((linear(m=-1), lib.q8_last_error())))
    t.start()
    t.join()
    assert seen[0][0] == ERR_SHAPE and b"m=-1" in seen[0][1]
    assert b"k=24" in lib.q8_last_error() and b"f8_linear" in lib.q8_last_error()
