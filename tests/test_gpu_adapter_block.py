"""The example that runs the operators together: training brings the block near its teacher, its
gradients are those of the loss, and decoding token by token gives the whole sequence's output."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def ab():
    from dora_adapter_linear_gb300.build import build
    build()
    import adapter_block
    return adapter_block


@pytest.mark.parametrize("bits", [8, 32])
def test_training_brings_the_block_near_its_teacher(ab, bits):
    block, teacher = ab.pair()
    losses = ab.train(block, teacher, steps=60, state_bits=bits)
    first, last = sum(losses[:5]) / 5, sum(losses[-5:]) / 5
    assert all(x == x for x in losses) and last < 0.5 * first, (first, last)


def test_block_gradients_are_the_losss(ab):
    """The adapters' gradients along the step to the teacher: the loss falls by what they say."""
    block, teacher = ab.pair()
    for n in block.B:       # part of the way, so that every A has a gradient too
        block.B[n].copy_(teacher.B[n] * 0.5)
    X = torch.randn(96, 512, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    pos = torch.arange(48, device="cuda").repeat(2)
    want = teacher.forward(X, pos, 2)[0].float()

    def loss():
        out, saved, _ = block.forward(X, pos, 2)
        return (out.float() - want).square().mean().double(), saved, out

    at, saved, out = loss()
    off = out.float() - want
    grads = block.backward(saved, pos, 2, (off * (2 / off.numel())).bfloat16())
    params, start = block.adapters(), [p.clone() for p in block.adapters()]
    for which in (0, 1):    # all A, then all B
        ways = [torch.randn(p.shape, generator=torch.Generator(device="cuda").manual_seed(9 + i), device="cuda") * 0.1
                * p.float().abs().mean() if i % 2 == which else torch.zeros_like(p, dtype=torch.float32)
                for i, p in enumerate(params)]
        # along the gradient, so that the loss moves by more than bf16 noise
        ways = [w.abs() * g.float().sign() for w, g in zip(ways, grads)]
        values = []
        for sign in (1.0, -1.0):
            for p, s, w in zip(params, start, ways):
                p.copy_(s + sign * w)
            values.append(loss()[0])
        moved = sum((g.double() * ((s + w).bfloat16().double() - (s - w).bfloat16().double())).sum()
                    for g, s, w in zip(grads, start, ways))
        for p, s in zip(params, start):
            p.copy_(s)
        assert float(values[0] - values[1]) == pytest.approx(float(moved), rel=0.1), which


def test_decoding_matches_the_whole_sequence(ab):
    block, teacher = ab.pair()
    X = torch.randn(3, 17, 512, generator=torch.Generator(device="cuda").manual_seed(4), device="cuda").bfloat16()
    whole = teacher.forward(X.reshape(51, 512), torch.arange(17, device="cuda").repeat(3), 3)[0].view(3, 17, 512)
    step = ab.decode(teacher, X, 3)
    # bf16 tensors between the calls: a few roundings of values of about 1 (largest about 4)
    assert float((step.float() - whole.float()).norm() / whole.float().norm()) < 1e-2
