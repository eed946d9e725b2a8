"""Numbers that a double holds and fp32 does not: the optimiser's arithmetic is fp32."""
import ctypes

import pytest
import torch

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300.build import build
from fake_runtime import fake  # noqa: F401

INVALID, AT = 1, 1 << 20


def step(lib, **hyper):
    h = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, lr_device=None)
    h.update(hyper)
    t, g = (L.LoraAdamwTensor * 1)(L.LoraAdamwTensor(AT, 1000, 1.0, 0.0, L.LORA_F32)), (ctypes.c_void_p * 1)(AT)
    state = L.LoraAdamwState(AT, AT, AT, AT, AT, AT, 32)
    return lib.adamw_step(t, g, 1, ctypes.byref(state), ctypes.byref(L.LoraAdamwHyper(**h)), None, None)


@pytest.mark.parametrize("hyper,status", [
    (dict(eps=1e-50), INVALID), (dict(eps=1e-40), INVALID), (dict(eps=2.0 ** -126), 0), (dict(eps=1e39), INVALID),
    (dict(lr=1e39), INVALID), (dict(lr=-1e39), INVALID), (dict(lr=1e38), 0), (dict(lr=1e-60), 0),
    (dict(grad_scale=1e39), INVALID), (dict(grad_scale=-1e300), INVALID), (dict(grad_scale=1e-30), 0), (dict(), 0),
])
def test_step_takes_what_fp32_holds(fake, hyper, status):  # noqa: F811
    assert step(fake, **hyper) == status


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_elements_without_a_gradient_stay(bits):
    build()
    from dora_adapter_linear_gb300 import optim
    p = torch.randn(3, 300, device="cuda:0")
    for eps in (1e-50, 1e-40, 1e39):
        with pytest.raises(ValueError, match="eps"):
            optim.AdamW([p], eps=eps)
    before = p.clone()
    opt = optim.AdamW([p], eps=2.0 ** -126, weight_decay=0.0, state_bits=bits)
    opt.step([torch.zeros_like(p)])
    assert torch.equal(p, before)
    for bad in (dict(lr=1e39), dict(grad_scale=1e39)):
        with pytest.raises(L.LoraError):
            opt.step([torch.zeros_like(p)], **bad)
    assert opt.steps == 1


@pytest.mark.parametrize("max_norm", [1e-50, 1e-46, 0.0, -1.0, float("nan")])
def test_a_clip_that_fp32_does_not_hold_is_refused(monkeypatch, max_norm):
    """It would be 0 in the kernels, where 0 stands for no clip."""
    from dora_adapter_linear_gb300 import optim
    opt = optim.AdamW.__new__(optim.AdamW)
    opt.params, opt._device = [torch.zeros(4)], torch.device("cpu")
    opt.lr, opt.betas, opt.eps, opt._tensors, opt._ws, opt._state = 1e-3, (0.9, 0.999), 1e-8, None, None, None
    monkeypatch.setattr(L, "host", lambda: type("Host", (), {"pair": lambda *a: torch.zeros(()), "pointers": lambda *a: b"",
                                                             "written": lambda *a: None}))
    for name in ("adamw_grad_norm", "adamw_step"):
        monkeypatch.setattr(L, name, lambda *a: None)
    opt.step([torch.zeros(4)], max_norm=1e-40)      # held, if with fewer bits
    with pytest.raises(ValueError, match="max_norm"):
        opt.step([torch.zeros(4)], max_norm=max_norm)
