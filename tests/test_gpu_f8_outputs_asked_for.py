"""Outputs that a caller asks for by True or by a tensor: what is neither is refused, not taken as True with the
caller's buffer left as it was."""

from __future__ import annotations

import numpy as np
import pytest

from f8_cases import inputs, to_dev, weight
from gpu_util import torch_dev

pytestmark = pytest.mark.gpu


def test_neither_a_truth_value_nor_a_tensor():
    torch, dev = torch_dev()
    import block_quantized_weight_linear_amd as q8
    rng = np.random.default_rng(1)
    wq, wd, xq, xd = to_dev(torch, dev, *weight(rng, 20, 160, parts=2)[:2], *inputs(rng, 4, 160)[:2])
    dx, dw, gu, dh = (torch.zeros(*s, device=dev) for s in ((4, 160), (40, 160), (4, 40), (4, 20)))
    dy, one = torch.ones(4, 40, device=dev), wd[:1]
    for wrong in ([dx], (dw,), "dx", {}, dx.cpu().numpy(), 2, object()):
        for call in (lambda **kw: q8.f8_linear_backward(wq, one, xq, xd, dy, **kw),
                     lambda **kw: q8.f8_linear_fused_gate_up_silu_backward(wq, wd, xq, xd, gu, dh, **kw)):
            for name in ("dx", "dw"):
                with pytest.raises(ValueError):
                    call(**{name: wrong})
        with pytest.raises(ValueError):
            q8.f8_linear_fused_gate_up_silu(wq, wd, xq, xd, keep_gate_up=wrong)
    for no, yes in ((False, True), (None, 1), (0, np.True_)):
        assert q8.f8_linear_backward(wq, one, xq, xd, dy, dx=no, dw=yes)[0] is None
        assert q8.f8_linear_backward(wq, one, xq, xd, dy, dx=yes, dw=no)[0].shape == (4, 160)
        assert torch.is_tensor(q8.f8_linear_fused_gate_up_silu(wq, wd, xq, xd, keep_gate_up=no))
        assert q8.f8_linear_fused_gate_up_silu(wq, wd, xq, xd, keep_gate_up=yes)[1].shape == (4, 40)
