"""The host side of the entry points on two devices, over a stand-in for the CUDA runtime (fake_cudart.cpp)."""
import ctypes

import pytest

from dora_adapter_linear_gb300 import _lib as L
from fake_runtime import fake  # noqa: F401

AT = 1 << 20        # never dereferenced
WS, SIZE = 1 << 30, 1 << 40


def norm_bwd(lib, dtype, M, D, per, post=1):
    sh = L.LoraNormShape(M, D, per, D, D, D, D, 1.0, 1e-6, 0.0, post, dtype)
    p = [AT] * 9 + [2 * AT] * 5
    if not post:
        p[3] = p[12] = None
    return lib.block_norm_bwd(ctypes.byref(sh), *p, WS, SIZE, None)


def linear(lib, r, backward):
    sh = L.shape(512, 1024, 2048, r, L.LORA_BF16)
    if backward:
        return lib.lora_linear_bwd(ctypes.byref(sh), *[AT] * 6, 1.0, *[AT] * 4, WS, SIZE, None)
    return lib.lora_linear_fwd(ctypes.byref(sh), *[AT] * 5, 1.0, AT, AT, WS, SIZE, None)


def norm_fwd(lib, dtype, M, D, per):
    sh = L.LoraNormShape(M, D, per, D, D, D, D, 1.0, 1e-6, 0.0, 1, dtype)
    return lib.block_norm_fwd(ctypes.byref(sh), *[AT] * 5, *[2 * AT] * 4, None)


CALLS = {
    "ring, two rows a barrier": lambda lib: norm_bwd(lib, L.LORA_BF16, 600, 4096, 1),
    "ring, two vectors": lambda lib: norm_bwd(lib, L.LORA_BF16, 600, 8192, 600),
    "ring, fp32": lambda lib: norm_bwd(lib, L.LORA_F32, 600, 4096, 100, post=0),
    "ring, pairs": lambda lib: norm_bwd(lib, L.LORA_F32, 600, 6144, 100),
    "short rows": lambda lib: norm_bwd(lib, L.LORA_BF16, 600, 1024, 100),
    "two passes": lambda lib: norm_bwd(lib, L.LORA_F32, 600, 16384, 100),
    "walk": lambda lib: norm_fwd(lib, L.LORA_BF16, 16384, 8192, 1),
    "linear forward": lambda lib: linear(lib, 64, False),
    "linear backward": lambda lib: linear(lib, 64, True),
    "dropout backward": lambda lib: lib.lora_linear_dropout_bwd(
        ctypes.byref(L.shape(512, 1024, 2048, 128, L.LORA_BF16)), AT, AT, 1.0, *[AT] * 5, 1.0, *[AT] * 4, WS, SIZE, None),
    "int8 product": lambda lib: lib.w8a8_lora_fwd(512, 1024, 2048, 16, *[AT] * 6, 1.0, *[AT] * 3, WS, SIZE, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_a_second_device_asks_for_its_shared_memory_there(fake, name):  # noqa: F811
    before = fake.fake_launches()
    for device in (0, 1, 0):
        fake.fake_device(device)
        assert CALLS[name](fake) == 0, device
    assert fake.fake_launches() >= before + 3
