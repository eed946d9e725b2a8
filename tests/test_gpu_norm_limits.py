"""The norm backward at the widths where one of its variants ends: four input rows or, with a gate row per row,
five have to fit the stages of a CTA or of a pair."""
import pytest
import torch

import test_gpu_block_ops as T
from test_gpu_block_ops import ops  # noqa: F401

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,D", [(BF16, 4096), (BF16, 4104), (BF16, 8192), (BF16, 8200), (BF16, 16384), (BF16, 16392),
                                     (F32, 3584), (F32, 3592), (F32, 4096), (F32, 4104), (F32, 8192), (F32, 8200)])
@pytest.mark.parametrize("gate", ["seq", "none"])
def test_four_inputs(ops, dtype, D, gate):  # noqa: F811
    T.test_norm(ops, 331, D, gate, True, dict(rpg=100) if gate == "seq" else {}, dtype)


@pytest.mark.parametrize("dtype,D", [(BF16, 4096), (BF16, 7640), (BF16, 7648), (BF16, 15280), (BF16, 15288), (BF16, 16384),
                                     (F32, 2864), (F32, 2872), (F32, 3816), (F32, 3824), (F32, 7632), (F32, 7640),
                                     (F32, 8192)])
@pytest.mark.parametrize("post", [True, False])
def test_five_inputs(ops, dtype, D, post):  # noqa: F811
    T.test_norm(ops, 331, D, "token", post, dict(alpha=0.22), dtype)
