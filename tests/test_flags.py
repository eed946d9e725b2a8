"""Flags whose truth raises: the error is the caller's to see, as it is raised."""
import pytest
import torch

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import ops


class NoTruth:
    def __bool__(self):
        raise KeyError("no truth")


X = torch.zeros(8, 32, dtype=torch.bfloat16)


@pytest.mark.parametrize("flag", ["pre_norm", "post_norm"])
def test_forward(flag):
    with pytest.raises(KeyError, match="no truth"):
        ops.block_norm_fwd(X, X, **{flag: NoTruth()})
    with pytest.raises(RuntimeError, match="ambiguous"):
        ops.block_norm_fwd(X, X, **{flag: torch.zeros(2)})


@pytest.mark.parametrize("at", [12, 13, 14, 15])
def test_backward(at):
    r = torch.ones(8)
    a = [X, X, r, r, X, X, None, None, None, None, 1.0, 0.0, False, True, True, True, torch.zeros(1024, dtype=torch.uint8)]
    assert L.host().block_norm_bwd(*a) is None          # CPU tensors are not for the native call
    a[at] = NoTruth()
    with pytest.raises(KeyError, match="no truth"):
        L.host().block_norm_bwd(*a)
