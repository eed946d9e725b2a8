"""Tensors that a call writes in place beside autograd: it notices the change of what it keeps for a backward."""
import pytest
import torch

DEV = "cuda:0"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def ops():
    from dora_adapter_linear_gb300.build import build
    build()
    from dora_adapter_linear_gb300 import ops as _ops
    return _ops


class NoHost:
    """Stands in for the host module: no call is for it."""

    def __getattr__(self, name):
        return lambda *a: None


def test_versions_of_an_optimisers_tensors(ops):
    """Only what has a gradient was written; a detached tensor shares its version with the parameter."""
    params = [torch.zeros(4, requires_grad=True) for _ in range(3)]
    tensors = [p.detach() for p in params] + [torch.inference_mode()(torch.zeros)(4)]
    addresses = b"".join(int(a).to_bytes(8, "little") for a in (4096, 0, 1 << 40, 64))
    ops.L.host().written(tensors, addresses)
    assert [p._version for p in params] == [1, 0, 1]
    assert ops.L.host().written(tensors, addresses[:-1]) is None and [p._version for p in params] == [1, 0, 1]


@pytest.mark.gpu
@pytest.mark.parametrize("native", [True, False])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotary_in_place_moves_the_version(ops, monkeypatch, native, inverse):
    if not native:
        monkeypatch.setattr(ops.L, "host", NoHost)
    call = ops.rotary_bwd if inverse else ops.rotary_fwd
    plan, pos = ops.rotary_plan(32, device=DEV), torch.arange(6, device=DEV)
    X, w = torch.randn(6, 2, 32, device=DEV), torch.ones(6, 2, 32, device=DEV, requires_grad=True)
    before = X._version
    kept = (X * w).sum()                    # autograd keeps X for the gradient of w
    out = torch.empty_like(X)
    call(X, pos, plan, out=out)
    assert X._version == before and out._version == 1 and call(X, pos, plan)._version == 0
    call(X, pos, plan, out=X)
    assert X._version == before + 1
    with pytest.raises(RuntimeError, match="inplace operation"):
        kept.backward()
    with torch.inference_mode():
        Y = torch.randn(6, 2, 32, device=DEV)
    call(Y, pos, plan, out=Y)               # has no version to move


@pytest.mark.gpu
def test_a_step_moves_its_parameters_versions(ops):
    from dora_adapter_linear_gb300 import optim
    params = [torch.randn(5, 8, device=DEV, requires_grad=True) for _ in range(3)]
    opt = optim.AdamW(params)
    x = torch.randn(5, 8, device=DEV, requires_grad=True)
    kept = [(x * p).sum() for p in params]
    grads = [torch.ones_like(p) for p in params]
    before = [p._version for p in params]
    opt.step([grads[0], None, grads[2]], max_norm=1.0)
    assert [p._version - b for p, b in zip(params, before)] == [1, 0, 1]
    for i in (0, 2):
        with pytest.raises(RuntimeError, match="inplace operation"):
            kept[i].backward()
    kept[1].backward()
    with pytest.raises(ops.L.LoraError):
        opt.step(grads, lr=float("nan"))    # refused: nothing was written
    assert [p._version - b for p, b in zip(params, before)] == [1, 0, 1]


def test_rotary_into_a_tensor_that_needs_a_gradient_is_refused(ops):
    plan, pos = ops.rotary_plan(32, device="cpu"), torch.arange(6)
    out = torch.zeros(6, 2, 32, requires_grad=True)
    for call in (ops.rotary_fwd, ops.rotary_bwd):
        with pytest.raises(ValueError, match="gradient"):
            call(torch.zeros(6, 2, 32), pos, plan, out=out)


@pytest.mark.gpu
def test_rotary_into_a_tensor_that_needs_a_gradient(ops):
    plan, pos = ops.rotary_plan(32, device=DEV), torch.arange(6, device=DEV)
    W = torch.randn(64, 64, device=DEV, requires_grad=True)
    X = torch.randn(6, 64, device=DEV) @ W
    heads = X.view(6, 2, 32)
    before = heads.detach().clone()
    for call in (ops.rotary_fwd, ops.rotary_bwd):
        with pytest.raises(ValueError, match="gradient"):
            call(heads, pos, plan, out=heads)
        assert torch.equal(heads, before)
    with torch.no_grad():
        assert ops.rotary_fwd(heads, pos, plan, out=heads) is heads
    assert not torch.equal(heads, before)
    ops.rotary_fwd(before, pos, plan, out=before)
    assert torch.equal(heads, before)
