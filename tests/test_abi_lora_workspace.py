"""Workspace sizes of the packed adapter calls, on the host (no GPU needed): one row on the
one-row kernel needs room for the adapter's inner products alone."""

from __future__ import annotations

import pytest

q8 = pytest.importorskip("block_quantized_weight_linear_amd")


@pytest.mark.parametrize("n,k,rank,ns", [(64, 256, 8, 1), (6144, 4096, 16, 3), (1 << 20, 16384, 256, 4)])
def test_one_row_needs_no_product(n, k, rank, ns):
    assert q8.q8_linear_lora_workspace_bytes(1, n, k, rank, ns) == q8.lora_workspace_bytes(1, rank, ns)


def test_the_other_forms_need_theirs():
    # past the one-row kernel's width, and from 256 rows on: the shared product of a fused matrix
    assert q8.q8_linear_lora_workspace_bytes(1, 6144, 16640, 16) >= 4 * 6144
    assert q8.q8_linear_lora_workspace_bytes(256, 6144, 4096, 16) >= 4 * 256 * 6144
    # two rows: their digits
    assert q8.q8_linear_lora_workspace_bytes(2, 64, 4096, 16) >= 4 * 2 * 4096
