"""Calls whose operands are on another device than the current one are refused before anything is launched.
The tensors are made up (shapes and devices without memory), so no second device is needed."""
import pytest
import torch
from torch._subclasses import fake_tensor
from torch._subclasses.fake_tensor import FakeTensorMode

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import ops, optim
from dora_adapter_linear_gb300.rotary import RotaryPlan

BF16, F32 = torch.bfloat16, torch.float32


class NoHost:
    """Stands in for the host module: no call is for it."""

    def __getattr__(self, name):
        return lambda *a: None


@pytest.fixture(autouse=True)
def no_context_of_a_made_up_device(monkeypatch):
    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda device: None, raising=False)


@pytest.fixture
def without_gpu(monkeypatch):
    monkeypatch.setattr(L, "current_device", lambda: 0, raising=False)
    monkeypatch.setattr(L, "host", NoHost)

    def launched(*a, **k):
        raise AssertionError("a call reached the library")
    for name in ("block_norm_fwd", "block_norm_bwd", "rotary_fwd", "rotary_bwd", "adamw_step", "adamw_grad_norm",
                 "adamw_fill_master", "dora_rownorm2", "dora_colnorm2", "w8a8_quantize_rows", "lora_linear_fwd"):
        monkeypatch.setattr(L, name, launched)


def elsewhere(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype, device="cuda:1")


def calls():
    """Each a call with every operand on cuda:1."""
    t = elsewhere
    plan = RotaryPlan(t(4, dtype=torch.int64), 8, 1.0, 0)
    return {
        "norm forward": lambda: ops.block_norm_fwd(t(8, 32), t(8, 32)),
        "norm backward": lambda: ops.block_norm_bwd(t(8, 32), t(8, 32), t(8, dtype=F32), None, t(8, 32), t(8, 32)),
        "rotary forward": lambda: ops.rotary_fwd(t(6, 2, 32), t(6, dtype=torch.int64), plan),
        "rotary backward": lambda: ops.rotary_bwd(t(6, 2, 32), t(6, dtype=torch.int64), plan),
        "optimiser": lambda: optim.AdamW([t(4, 4)]),
        "workspace": lambda: ops.workspace(1024, torch.device("cuda", 1)),
        "linear": lambda: ops.lora_linear_fwd(t(8, 32), t(16, 32), t(8, 32), t(16, 8), 1.0),
        "row norms": lambda: ops.dora_rownorm2(t(8, 32)),
        "column norms": lambda: ops.dora_colnorm2(t(8, 32)),
        "quantiser": lambda: ops.w8a8_quantize_rows(t(8, 32)),
    }


@pytest.mark.parametrize("name", ["norm forward", "norm backward", "rotary forward", "rotary backward", "optimiser",
                                  "workspace", "linear", "row norms", "column norms", "quantiser"])
def test_refused_by_the_wrappers(without_gpu, name):
    with FakeTensorMode():
        call = calls()[name]
        with pytest.raises(ValueError, match="current device"):
            call()


def test_a_step_under_another_device_is_refused(without_gpu, monkeypatch):
    opt = optim.AdamW.__new__(optim.AdamW)      # one that was made while its device was the current one
    with FakeTensorMode():
        opt.params, opt._device = [elsewhere(4, 4)], torch.device("cuda", 1)
        monkeypatch.setattr(optim.AdamW, "_pointers", lambda self, grads: pytest.fail("the step went on"))
        with pytest.raises(ValueError, match="current device"):
            opt.step([elsewhere(4, 4)])


def test_workspace_sizes_are_of_a_device(without_gpu, monkeypatch):
    """A larger device has more parts, and each of them partial sums of its own."""
    current, asked = [0], []
    monkeypatch.setattr(L, "current_device", lambda: current[0])
    monkeypatch.setattr(L, "block_norm_bwd_workspace_bytes", lambda sh: (1 + current[0]) << 20)
    monkeypatch.setattr(ops, "workspace", lambda nbytes, device: asked.append(nbytes))
    monkeypatch.setattr(L, "block_norm_bwd", lambda *a: None)
    monkeypatch.setattr(L, "host", lambda: type("Host", (), {"block_norm_bwd": lambda *a: (None,) * 5}))
    for current[0] in (0, 1, 0):
        with FakeTensorMode():
            t = lambda *s, dtype=BF16: torch.zeros(*s, dtype=dtype, device=f"cuda:{current[0]}")  # noqa: B023,E731
            ops.block_norm_bwd(t(9, 48), t(9, 48), t(9, dtype=F32), None, t(9, 48), t(9, 48))
    assert asked == [1 << 20, 2 << 20, 1 << 20]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["norm forward", "norm backward", "rotary forward", "rotary backward"])
def test_refused_by_the_native_calls(name):
    from dora_adapter_linear_gb300.build import build
    build()
    torch.zeros(1, device="cuda:0")
    t = elsewhere
    host = L.host()
    with FakeTensorMode():
        if name == "norm forward":
            got = host.block_norm_fwd(t(8, 32), t(8, 32), None, None, None, None, 1.0, 1e-6, 0.0, True, False)
        elif name == "norm backward":
            got = host.block_norm_bwd(t(8, 32), t(8, 32), t(8, dtype=F32), None, t(8, 32), t(8, 32), None, None, None, None,
                                      1.0, 0.0, False, True, True, True, t(1 << 16, dtype=torch.uint8))
        else:
            got = host.rotary(name == "rotary backward", t(6, 2, 32), t(6, dtype=torch.int64), t(4, dtype=torch.int64), 8,
                              1.0, 0, None)
        assert got is None                      # left to the wrapper,
        with pytest.raises(ValueError, match="current device"):
            calls()[name]()                     # which names the fault
