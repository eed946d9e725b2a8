"""Every width of the block norm comes to its launches with the shared memory that it takes (over a stand-in for the
CUDA runtime), and the widths where that is just below 48 KB run."""
import ctypes

import pytest
import torch

from dora_adapter_linear_gb300 import _lib as L
from fake_runtime import fake  # noqa: F401

AT = 1 << 20        # never dereferenced
WS, SIZE = 1 << 30, 1 << 40


def calls(lib, dtype, M, D, per):
    sh = L.LoraNormShape(M, D, per, D, D, D, D, 1.0, 1e-6, 0.0, 1, dtype)
    return (lib.block_norm_fwd(ctypes.byref(sh), *[AT] * 5, *[2 * AT] * 4, None),
            lib.block_norm_bwd(ctypes.byref(sh), *[AT] * 9, *[2 * AT] * 5, WS, SIZE, None))


@pytest.mark.parametrize("dtype", [L.LORA_BF16, L.LORA_F32])
@pytest.mark.parametrize("per", [1, 100, 1 << 20])
def test_every_width(fake, dtype, per):  # noqa: F811
    """Each on a device of its own, so that no earlier width has asked for the same kernel there."""
    refused = []
    for D in range(8, 8200, 8):
        fake.fake_device(1000 + D)
        if calls(fake, dtype, 16384, D, per) != (0, 0):
            refused.append(D)
    fake.fake_device(0)
    assert not refused


@pytest.mark.gpu
@pytest.mark.parametrize("M,D,gate,dtype", [
    (400, 4096, "token", torch.bfloat16), (400, 4056, "token", torch.bfloat16), (300, 6144, "none", torch.bfloat16),
    (300, 6088, "row", torch.bfloat16), (900, 680, "none", torch.bfloat16), (900, 680, "row", torch.bfloat16),
    (900, 552, "token", torch.bfloat16), (900, 552, "token", torch.float32),
])
@pytest.mark.parametrize("post", [True, False])
def test_widths_just_below_48_kb(M, D, gate, dtype, post):
    import test_gpu_block_ops as T
    from dora_adapter_linear_gb300 import ops
    from dora_adapter_linear_gb300.build import build
    build()
    T.test_norm(ops, M, D, gate, post, {}, dtype)
