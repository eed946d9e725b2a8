"""Frequencies of the rotary positions: laid out once per model, kept on the device."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

from . import _lib as L

LAYOUTS = {"half": L.LORA_ROTARY_HALF, "interleaved": L.LORA_ROTARY_INTERLEAVED}


@dataclass(frozen=True)
class RotaryPlan:
    """freq: [rot_dim / 2] fractions of a turn per position in units of 2^-64 (int64 bit patterns), from fp64
    arithmetic: within 1.5 2^-53 of theta_j / (2 pi) and half a unit;
    scale: factor on the rotated values; layout: the C ABI's lora_rotary_layout."""
    freq: torch.Tensor
    rot_dim: int
    scale: float
    layout: int


def rotary_angles(rot_dim, base=10000.0, scaling="none", factor=1.0, original=8192, low=1.0, high=4.0, beta_fast=32.0,
             beta_slow=1.0):
    """Angles per position theta_j, j < rot_dim / 2 (fp64), and the factor on the rotated values.
      none    theta_j = base^(-2 j / rot_dim)
      linear  theta_j / factor: positions interpolated
      ntk     base raised by factor^(rot_dim / (rot_dim - 2)): the longest wave stretched by factor
      bands   by turns over the original context, original theta_j / (2 pi): above `high` kept, below
              `low` divided by factor, linear in the turns between
      yarn    the same with a ramp over j between the pairs that make beta_fast and beta_slow turns;
              rotated values times 0.1 ln(factor) + 1"""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not base > 1.0 or not factor >= 1.0 or not original > 0:
        raise ValueError("base must be above 1, factor at least 1 and original above 0")
    half, scale = rot_dim // 2, 1.0
    if scaling == "ntk":
        base = base * factor ** (rot_dim / max(rot_dim - 2, 1))
    theta = [base ** (-2 * j / rot_dim) for j in range(half)]
    if scaling == "linear":
        theta = [t / factor for t in theta]
    elif scaling == "bands":
        if not high > low:
            raise ValueError("high must be above low")
        keep = [min(max((original * t / (2 * math.pi) - low) / (high - low), 0.0), 1.0) for t in theta]
        theta = [(1 - k) * t / factor + k * t for k, t in zip(keep, theta)]
    elif scaling == "yarn":
        def pair(turns):
            return rot_dim * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base))
        first, last = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), rot_dim - 1)
        width = last - first if last > first else 0.001
        ramp = [min(max((j - first) / width, 0.0), 1.0) for j in range(half)]
        theta = [r * t / factor + (1 - r) * t for r, t in zip(ramp, theta)]
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in ("none", "ntk"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return torch.tensor(theta, dtype=torch.float64), scale


def rotary_plan(rot_dim, base=10000.0, layout="half", scaling="none", inv_freq=None, scale=None, device="cuda",
                **how):
    """A RotaryPlan for rotary_fwd / rotary_bwd.  layout: "half" pairs (j, j + rot_dim / 2),
    "interleaved" pairs (2 j, 2 j + 1).  The angles per position come from rotary_angles() (`base`,
    `scaling` and its parameters) or are given as inv_freq [rot_dim / 2]; `scale` replaces the factor
    on the rotated values."""
    if layout not in LAYOUTS:
        raise ValueError(f"unknown layout {layout!r}")
    if inv_freq is None:
        theta, own_scale = rotary_angles(rot_dim, base, scaling, **how)
    else:
        if scaling != "none" or how:
            raise ValueError("a given inv_freq is used as it is: no scaling parameters beside it")
        theta, own_scale = inv_freq.detach().to("cpu", torch.float64), 1.0
        if rot_dim < 2 or tuple(theta.shape) != (rot_dim // 2,) or rot_dim % 2 or not bool(theta.isfinite().all()):
            raise ValueError(f"inv_freq must be [{rot_dim // 2}] finite angles per position")
    scale = own_scale if scale is None else float(scale)
    if not math.isfinite(scale):
        raise ValueError("scale must be finite")
    bits = [round(t / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for t in theta.tolist()]
    freq = torch.tensor([b - 2 ** 64 if b >= 2 ** 63 else b for b in bits], dtype=torch.int64, device=device)
    return RotaryPlan(freq, rot_dim, scale, LAYOUTS[layout])
