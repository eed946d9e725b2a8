"""Where a rotary call's output may lie: every placement that shares an element with the input is refused, every
other one goes on to its launch (over a stand-in for the CUDA runtime)."""
import ctypes
import random
import time

import pytest

from dora_adapter_linear_gb300 import _lib as L
from fake_runtime import fake  # noqa: F401

AT, INVALID = 1 << 40, 1


def call(lib, M, H, hd, x, y, d, dtype=L.LORA_BF16):
    """x, y: (token stride, head stride); d: how many elements after X's first one Y begins."""
    sh = L.LoraRotaryShape(M, H, hd, 2, *x, *y, 1.0, 0, 64, dtype)
    return lib.rotary_fwd(ctypes.byref(sh), AT, 8, 8, AT + d * (4 if dtype == L.LORA_F32 else 2), None)


def elements(M, H, hd, strides, d=0):
    return [d + i * strides[0] + h * strides[1] + c for i in range(M) for h in range(H) for c in range(hd)]


def test_small_placements_against_every_element(fake):  # noqa: F811
    rng = random.Random(5)
    seen = {True: 0, False: 0, "itself": 0}
    for _ in range(20000):
        M, H, hd = rng.choice((1, 2, 3, 5)), rng.choice((1, 2, 3, 4)), rng.choice((2, 3, 4))
        inner = hd + rng.randrange(5)
        rows = (inner * (H - 1) + hd + rng.choice((0, 1, hd, 3 * hd, H * inner)), inner)        # tokens outside
        inner = hd + rng.randrange(5)
        heads = (inner, inner * (M - 1) + hd + rng.choice((0, 2, hd, M * inner)))               # heads outside
        free = (rng.randrange(3 * H * hd), rng.randrange(2 * hd))
        x, y = rng.choice((rows, heads, free)), rng.choice((rows, rows, heads, free))
        if rng.random() < 0.3:
            y = (x[0], y[1])
        d = rng.randrange(-2 * M * H * hd, 2 * M * H * hd + 1) or 1
        ys = elements(M, H, hd, y, d)
        status = call(fake, M, H, hd, x, y, d, rng.choice((L.LORA_BF16, L.LORA_F32)))
        if len(set(ys)) < len(ys):
            seen["itself"] += 1
            assert status == INVALID, (M, H, hd, x, y, d)
            continue
        meet = not set(ys).isdisjoint(elements(M, H, hd, x))
        seen[meet] += 1
        # rows of y that reach into one another without a common element are no layout that the call takes
        if status == INVALID and not meet:
            by_token = (H <= 1 or y[1] >= hd) and (M <= 1 or y[0] >= (H - 1) * y[1] + hd)
            by_head = (M <= 1 or y[0] >= hd) and (H <= 1 or y[1] >= (M - 1) * y[0] + hd)
            assert not by_token and not by_head, (M, H, hd, x, y, d)
        else:
            assert status == (INVALID if meet else 0), (M, H, hd, x, y, d)
    assert min(seen.values()) > 1000, seen


@pytest.mark.parametrize("M", [1, 16384, (1 << 31) - 1])
def test_columns_of_one_packed_projection(fake, M):  # noqa: F811
    """Query heads turned into the place of other columns, of as many tokens as there may be, at once."""
    H, hd, row = 40, 128, 96 * 128
    begin = time.perf_counter()
    for d, status in ((40 * hd, 0), (56 * hd, 0), (39 * hd, INVALID), (1, INVALID), (-1, INVALID), (row - hd, 0 if M == 1 else
                      INVALID), (row * M, 0), (56 * hd + 1, 0 if M == 1 else INVALID)):
        assert call(fake, M, H, hd, (row, hd), (row, hd), d) == status, d
    # every other head of the same columns
    assert call(fake, M, H, hd, (row, 2 * hd), (row, 2 * hd), hd) == 0
    assert call(fake, M, H, hd, (row, 2 * hd), (row, 2 * hd), hd - 1) == INVALID
    # [heads, tokens, head_dim] beside itself
    assert call(fake, M, H, hd, (hd, M * hd), (hd, M * hd), M * H * hd) == 0
    assert call(fake, M, H, hd, (hd, M * hd), (hd, M * hd), M * H * hd - 1) == INVALID
    # one head read by every token, into rows beside it
    assert call(fake, M, H, hd, (0, hd), (row, hd), H * hd) == 0
    assert call(fake, M, H, hd, (0, hd), (row, hd), -row * (M - 1) + hd) == INVALID
    assert time.perf_counter() - begin < 1.0
