"""Rotary plans: what a call takes of one, and the angles that its frequencies stand for."""
from dataclasses import replace

import pytest
import torch

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import ops


@pytest.mark.parametrize("change", [
    dict(rot_dim=16), dict(rot_dim=32), dict(freq=torch.zeros(3, dtype=torch.int64)), dict(freq=torch.zeros(4)),
    dict(freq=torch.zeros(8, dtype=torch.int64)[::2]), dict(freq=torch.zeros(4, 1, dtype=torch.int64)),
])
def test_a_plan_whose_frequencies_do_not_fit_is_refused(monkeypatch, change):
    """The kernel reads rot_dim / 2 of them."""
    monkeypatch.setattr(ops, "_need_cuda", lambda name, t: None)
    for name in ("rotary_fwd", "rotary_bwd"):
        monkeypatch.setattr(L, name, lambda *a: pytest.fail("the call reached the library"))
    plan = replace(ops.rotary_plan(8, device="cpu"), **change)
    for call in (ops.rotary_fwd, ops.rotary_bwd):
        with pytest.raises(ValueError, match="freq"):
            call(torch.zeros(6, 2, 32), torch.arange(6), plan)
