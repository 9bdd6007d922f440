"""The copy of the library's rules in f8_tiles.py against the library's own: the backward calls' by the workspace that
they ask for, the forward calls' by the numbers in their source (no GPU needed)."""

from __future__ import annotations

import os
import re

import numpy as np
import pytest

import f8_tiles
from block_quantized_weight_linear_amd import build

q8 = pytest.importorskip("block_quantized_weight_linear_amd")


@pytest.mark.parametrize("kind,type", [("float32", 0), ("float16", 1), ("bfloat16", 2)])
def test_backward_rules(kind, type):
    rng = np.random.default_rng(type)
    seen = set()
    for _ in range(400):
        m, n = (int(2 ** rng.uniform(0, 12)) for _ in range(2))
        k = 16 * int(2 ** rng.uniform(0, 9))
        for parts, fn in ((1, q8.lib.f8_linear_backward_workspace_bytes),
                          (2, q8.lib.f8_linear_fused_gate_up_silu_backward_workspace_bytes)):
            assert fn(m, n, k, type) == f8_tiles.backward_bytes(m, n, k, kind, parts), (m, n, k, parts)
            seen.add((f8_tiles.dx_form(m, n, k, kind, parts), f8_tiles.dw_form(m, n, k, kind, parts)))
    assert len(seen) >= 7, seen


def test_forward_rule():
    with open(os.path.join(build.CSRC, "f8_linear.hip")) as f:
        source = f.read()
    numbers = lambda what: re.search(re.escape(what) + r" = \{([^}]*)\}", source).group(1).split(", ")  # noqa: E731
    assert tuple(int(v) for v in numbers("bn[5]")) == f8_tiles.WEIGHT_ROWS
    assert "constexpr int BIG = WIDE ? 4 : 8;" in source and "constexpr bool THIRD = !WIDE && !SILU;" in source
    for width, big in (("wide", 4), ("narrow", 8)):
        assert tuple(32 * big if v == "32 * BIG" else int(v) for v in numbers("bm[5]")) == f8_tiles.ROWS[width]
        pick = [re.fullmatch(r"WIDE \? (\d+) : (\d+)", v) for v in numbers("cost[5]")]
        cost = [int(p.group(1 if width == "wide" else 2)) if p else int(v) for p, v in zip(pick, numbers("cost[5]"))]
        assert tuple(cost) == f8_tiles.COST[width]
    for m, n_out in ((65, 100), (300, 2001), (4096, 6144), (4097, 6140)):
        assert f8_tiles.forward_tile(m, n_out, "bfloat16", False) in zip(f8_tiles.WEIGHT_ROWS, f8_tiles.ROWS["narrow"])
