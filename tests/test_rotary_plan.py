"""Rotary plans: what a call takes of one, and the angles that its frequencies stand for."""
from dataclasses import replace
from decimal import Decimal, localcontext
from fractions import Fraction

import numpy as np
import pytest
import torch

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import ops
from dora_adapter_linear_gb300.rotary import rotary_angles


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


PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def turns(theta, pos):
    """The fraction of a turn that position pos makes at theta per position, within 2^-180 of a turn here."""
    return Fraction(theta) * pos / (2 * PI) % 1


def off(theta):
    """What a frequency may be off by, in turns: 2 pi and the quotient are rounded to fp64 (2^-54.5 and 2^-53),
    then the fraction to 64 bits."""
    return abs(Fraction(theta)) / (2 * PI) * Fraction(3, 2 ** 54) + Fraction(1, 2 ** 65)


def apart(a, b):
    """Of two fractions of a turn, the shorter way around."""
    d = abs(a - b) % 1
    return min(d, 1 - d)


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (96, 500000.0), (128, 1e6), (514, 1e4)])
@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "bands", "yarn"])
def test_frequencies_stand_for_the_angles(rot, base, scaling):
    """After p positions the angle is off by p times what fp64 and the fraction's last bit leave, up to the last one."""
    how = {} if scaling == "none" else dict(factor=8.0)
    theta, _ = rotary_angles(rot, base, scaling, **how)
    plan = ops.rotary_plan(rot, base, scaling=scaling, device="cpu", **how)
    for pos in (1, 131072, 1 << 31, 1 << 40, (1 << 63) - 1, -(1 << 63)):
        for t, f in zip(theta.tolist(), plan.freq.tolist()):
            assert apart(Fraction(f * pos % 2 ** 64, 2 ** 64), turns(t, pos)) <= abs(pos) * off(t)


@pytest.mark.parametrize("theta", [0.0, -1.0, 1.0, 6.283185307179586, 1e-300, 5e-324, 12345.678, -3e20, 1e40])
def test_frequencies_of_any_angle(theta):
    plan = ops.rotary_plan(2, inv_freq=torch.tensor([theta], dtype=torch.float64), device="cpu")
    f = Fraction(plan.freq.item() % 2 ** 64, 2 ** 64)
    assert apart(f, turns(theta, 1)) <= off(theta)


@pytest.mark.parametrize("rot,base", [(96, 500000.0), (128, 10000.0)])
def test_angles_are_those_of_the_formula(rot, base):
    """fp64: the power within 2 units of its last place."""
    theta, _ = rotary_angles(rot, base)
    with localcontext() as ctx:
        ctx.prec = 60
        for j, t in enumerate(theta.tolist()):
            exact = Decimal(base) ** (Decimal(-2 * j) / rot)
            # the exponent -2 j / rot is rounded too: 2^-53 of up to ln(base)
            assert abs(Decimal(t) - exact) <= exact * Decimal(2) ** -53 * (2 + Decimal(base).ln())


@pytest.mark.gpu
@pytest.mark.parametrize("longest", [1 << 17, 1 << 24, 1 << 31, 1 << 40])
def test_turned_heads_against_the_angles_themselves(longest):
    """Not against the plan's own fractions: the reference is the fp64 angle, exactly reduced."""
    from dora_adapter_linear_gb300.build import build
    build()
    rot, base = 96, 500000.0
    gen = torch.Generator().manual_seed(longest % 1000)
    pos = torch.randint(longest // 2, longest, (40,), generator=gen)
    x = torch.randn(40, 3, rot, generator=gen)
    theta, _ = rotary_angles(rot, base)
    angle = np.array([[float(turns(t, int(p))) * 2 * np.pi for t in theta.tolist()] for p in pos.tolist()])
    got = ops.rotary_fwd(x.cuda(), pos.cuda(), ops.rotary_plan(rot, base)).double().cpu().numpy()
    a, b = (x[..., :rot // 2].double().numpy(), x[..., rot // 2:].double().numpy())
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    ref = np.concatenate((a * c - b * s, b * c + a * s), -1)
    both = np.concatenate((np.abs(a) + np.abs(b),) * 2, -1)
    # 8 fp32 roundings of the terms and one of the store, and what the frequencies (theta <= 1) are off by
    assert (np.abs(got - ref) <= (9 * 2.0 ** -24 + longest * 2 * np.pi * float(off(1.0))) * both).all()
