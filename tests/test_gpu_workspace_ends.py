"""The adapter calls and the MoE layer stay within a workspace of exactly the size they ask
for, whatever lies before and behind it, and give the same bits in it."""

from __future__ import annotations

import pytest

import workloads as wl
from gpu_util import say, to_dev, torch_dev
from test_gpu_lora import Case
from test_gpu_moe_layer import layer

pytestmark = pytest.mark.gpu

FENCE = 4096


@pytest.fixture(scope="module")
def q8():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8mod
    return q8mod, torch, dev


def fenced(env, size, call, what):
    """call(workspace) in the middle of a buffer; what lies around it stays as it was."""
    _, torch, dev = env
    say(f"{what}: {size} bytes")
    buf = torch.full((FENCE + size + FENCE,), 0xA5, dtype=torch.uint8, device=dev)
    got, want = call(buf[FENCE:FENCE + size]), call(None)
    assert (buf[:FENCE] == 0xA5).all() and (buf[FENCE + size:] == 0xA5).all(), what
    assert torch.equal(got, want), what


# every form of the packed calls: one row, tiles with and without a cut k, separate launches
@pytest.mark.parametrize("m,n,k,rank,sections", [(1, 130, 4096, 16, [100, 30]), (1, 64, 16640, 8, None),
                                                 (2, 34, 256, 8, None), (9, 100, 1024, 256, [50, 50]),
                                                 (31, 200, 8192, 16, None), (255, 66, 4352, 24, [1, 65]),
                                                 (256, 96, 512, 16, None), (300, 64, 1280, 64, [32, 32])])
def test_packed_calls(q8, m, n, k, rank, sections):
    lib, torch, dev = q8
    c = Case(q8, 7000 + m, m, n, k, 3, rank, "bfloat16", sections)
    w = to_dev(wl.q8_weight(7001, n, k)[0], dev)
    size = lib.q8_linear_lora_workspace_bytes(m, n, k, rank, len(c.parts))
    fenced(q8, size, lambda ws: lib.q8_linear_lora(w, n, k, c.xd, *c.args, **c.more, workspace=ws), f"linear m={m}")
    fenced(q8, size, lambda ws: lib.q8_linear_fused_gate_up_silu_lora(w, n // 2, k, c.xd, *c.args, **c.more, workspace=ws),
           f"gate_up m={m}")


@pytest.mark.parametrize("m,n,k", [(256, 96, 512), (300, 64, 1280), (2, 34, 16640)])
def test_plain_call_without_room_for_a_product(q8, m, n, k):
    lib, torch, dev = q8
    c = Case(q8, 7050 + m, m, n, k, 3, 16, "float16", None)
    w = to_dev(wl.q8_weight(7051, n, k)[0], dev)
    fenced(q8, lib.lora_workspace_bytes(m, 16), lambda ws: lib.q8_linear_lora(w, n, k, c.xd, *c.args, **c.more, workspace=ws),
           f"linear m={m}")


@pytest.mark.parametrize("m,n,k,count,rank", [(1, 70, 256, 2, 8), (47, 66, 512, 3, 16), (300, 64, 512, 4, 256),
                                              (48, 130, 8192, 2, 256), (1300, 58, 256, 256, 256), (700, 514, 512, 40, 64)])
def test_beside(q8, m, n, k, count, rank):
    lib, torch, dev = q8
    c = Case(q8, 7100 + m, m, n, k, count, rank, "float32")
    y = to_dev(wl.activations(7101, m, n), dev)
    size = lib.lora_workspace_bytes(m, rank)
    fenced(q8, size, lambda ws: lib.lora_add(y, c.xd, *c.args, **c.more, workspace=ws), f"lora_add m={m}")
    fenced(q8, size, lambda ws: lib.lora_gate_up_silu(y, c.xd, *c.args, **c.more, workspace=ws), f"lora_gate_up_silu m={m}")


@pytest.mark.parametrize("m,e,k,f,h", [(1, 8, 2, 256, 512), (60, 60, 4, 512, 256), (128, 128, 7, 256, 256),
                                       (129, 128, 3, 256, 256), (70, 8, 2, 256, 512), (3, 2, 1, 6144, 256)])
def test_moe_layer(q8, m, e, k, f, h):
    lib, torch, dev = q8
    gu, dn, wr = (to_dev(v, dev) for v in layer(7200, e, f, h))
    x = to_dev(wl.activations(7201, m, h), dev)
    fenced(q8, lib.q8_moe_layer_workspace_bytes(m, k, e, f, h),
           lambda ws: lib.q8_moe_layer(wr, gu, dn, e, f, h, x, k, workspace=ws), f"moe layer m={m}")
