"""Workspace sizes of the packed adapter calls, on the host (no GPU needed; nothing below
reaches a kernel): room only for what a call's form keeps there."""

from __future__ import annotations

import pytest

q8 = pytest.importorskip("block_quantized_weight_linear_amd")
from block_quantized_weight_linear_amd._binding import _Lora  # noqa: E402

ERR_WORKSPACE = 4


@pytest.mark.parametrize("n,k,rank,ns", [(64, 256, 8, 1), (6144, 4096, 16, 3), (1 << 20, 16384, 256, 4)])
def test_one_row_needs_no_product(n, k, rank, ns):
    assert q8.q8_linear_lora_workspace_bytes(1, n, k, rank, ns) == q8.lora_workspace_bytes(1, rank, ns)


def test_the_other_forms_need_theirs():
    # past the one-row kernel's width, and from 256 rows on: the shared product of a fused matrix
    assert q8.q8_linear_lora_workspace_bytes(1, 6144, 16640, 16) >= 4 * 6144
    assert q8.q8_linear_lora_workspace_bytes(256, 6144, 4096, 16) >= 4 * 256 * 6144
    # two rows: their digits
    assert q8.q8_linear_lora_workspace_bytes(2, 64, 4096, 16) >= 4 * 2 * 4096


@pytest.mark.parametrize("m,n,k", [(256, 6144, 4096), (2048, 64, 256), (2, 64, 16640), (200, 493504, 4096)])
def test_the_plain_call_keeps_no_product(m, n, k):
    """Where its product is q8_linear's, it goes straight into y (the fused call's has to wait
    for the activation): lora_add's workspace is enough, a byte less is refused."""
    fake, need = 0x10000, q8.lora_workspace_bytes(m, 16, 1)
    lo = _Lora(fake, fake, None, None, fake, (n,), 2, 3, 16, 1)
    assert q8.lib.q8_linear_lora(fake, n, k, fake, m, k, lo, fake, n, fake, need - 1, None) == ERR_WORKSPACE
    assert f"required {need}".encode() in q8.lib.q8_last_error()
    lo = _Lora(fake, fake, None, None, fake, (2 * n,), 2, 3, 16, 1)
    fused = q8.q8_linear_lora_workspace_bytes(m, 2 * n, k, 16)
    assert fused >= need + 8 * m * n
    assert q8.lib.q8_linear_fused_gate_up_silu_lora(fake, n, k, fake, m, k, lo, fake, n, fake, fused - 1,
                                                    None) == ERR_WORKSPACE
    assert f"required {fused}".encode() in q8.lib.q8_last_error()
