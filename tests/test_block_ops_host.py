"""Block norm, rotary positions and AdamW on the CPU: the fp64 reference against differences and
PyTorch, the rotary frequencies, and every refusal of the Python wrappers and the C ABI (nothing is
launched)."""
import ctypes
import math

import numpy as np
import pytest
import torch

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import ops, optim
from dora_adapter_linear_gb300.build import build
from dora_adapter_linear_gb300.rotary import rotary_angles
from oracle import block_oracle as BO


@pytest.fixture(scope="module")
def lib():
    build()
    return L._lib()


# ------------------------------------------------------------------ the reference itself
def _norm_case(seed, M=6, D=16, rpg=2, post=True, gate=True, y=True):
    r = np.random.default_rng(seed)
    n = r.standard_normal
    kw = dict(w_pre=1 + 0.1 * n(D), w_post=1 + 0.1 * n(D) if post else None,
              gate=n((-(-M // rpg), D)) if gate else None, rows_per_gate=rpg, alpha=0.7, off=0.25, post=post)
    return n((M, D)), n((M, D)) if y else None, kw, n((M, D)), n((M, D))


@pytest.mark.parametrize("post,gate,rpg", [(True, True, 2), (True, True, 4), (True, False, 1), (False, True, 1),
                                           (False, False, 1)])
def test_norm_reference_gradients_match_differences(post, gate, rpg):
    x, y, kw, dh, dz = _norm_case(1, rpg=rpg, post=post, gate=gate)
    z, _, r_pre, r_post = BO.block_norm_fwd(x, y, **kw)
    got = BO.block_norm_bwd(z, y, r_pre, r_post, dh, dz, **kw)

    def loss(x, y, **over):
        z, h, _, _ = BO.block_norm_fwd(x, y, **{**kw, **over})
        return (z * dz).sum() + (h * dh).sum()

    for name, value, grad in (("x", x, got[0]), ("y", y, got[1]), ("w_pre", kw["w_pre"], got[2]),
                              ("w_post", kw["w_post"], got[3]), ("gate", kw["gate"], got[4])):
        if value is None:
            continue
        v = np.random.default_rng(7).standard_normal(value.shape)
        at = lambda s: {name: value + s * 1e-5 * v}  # noqa: E731
        call = lambda s: loss(**{"x": x, "y": y, **at(s)})  # noqa: E731
        assert (call(1) - call(-1)) / 2e-5 == pytest.approx((grad * v).sum(), rel=1e-6, abs=1e-7), name


def test_norm_reference_matches_autograd_without_a_block_output():
    x, _, kw, dh, _ = _norm_case(2, y=False, post=False, gate=False)
    t = torch.from_numpy(x).requires_grad_(True)
    h = t * torch.rsqrt(t.pow(2).mean(1, keepdim=True) + 1e-6) * torch.from_numpy(kw["w_pre"] + kw["off"])
    h.backward(torch.from_numpy(dh))
    z, h64, r, _ = BO.block_norm_fwd(x, None, **kw)
    assert z is x and np.allclose(h64, h.detach().numpy(), rtol=1e-12)
    dx = BO.block_norm_bwd(z, None, r, None, dh, None, **kw)[0]
    assert np.allclose(dx, t.grad.numpy(), rtol=1e-10, atol=1e-12)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_reference_is_a_turn(layout):
    r = np.random.default_rng(3)
    x, turns = r.standard_normal((5, 3, 12)), r.uniform(-2, 2, (5, 4))
    y = BO.rotary(x, turns, layout)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose(BO.rotary(y, turns, layout, inverse=True), x)
    g = r.standard_normal(y.shape)      # the inverse is the transpose: <R x, g> = <x, R' g>
    assert (BO.rotary(x, turns, layout, 1.5) * g).sum() == pytest.approx((x * BO.rotary(g, turns, layout, 1.5, True)).sum())
    i, j = (0, 4) if layout == "half" else (0, 1)
    quarter = BO.rotary(x, np.full((5, 4), 0.25), layout)
    assert np.allclose(quarter[..., i], -x[..., j]) and np.allclose(quarter[..., j], x[..., i])


def test_adamw_reference_matches_torch():
    torch.manual_seed(4)
    p = torch.randn(40, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    q, m, v = p.detach().numpy().copy(), np.zeros(40), np.zeros(40)
    for t in range(1, 6):
        p.grad = torch.randn(40, dtype=torch.float64)
        opt.step()
        q, m, v = BO.adamw(q, p.grad.numpy(), m, v, t, 0.01, (0.8, 0.95), 1e-6, 0.1)
        assert np.allclose(q, p.detach().numpy(), rtol=1e-12)


# ------------------------------------------------------------------ rotary frequencies
def test_rotary_angles():
    plain, one = rotary_angles(64, 500000.0)
    assert one == 1.0 and plain[0] == 1.0 and plain[-1].item() == pytest.approx(500000.0 ** (-62 / 64), rel=1e-14)
    assert torch.allclose(rotary_angles(64, 500000.0, "linear", 4.0)[0] * 4, plain, rtol=1e-14)
    ntk = rotary_angles(64, 500000.0, "ntk", 4.0)[0]
    assert ntk[0] == 1.0 and ntk[-1].item() == pytest.approx(plain[-1].item() / 4, rel=1e-12)
    for kind in ("bands", "yarn"):
        f, scale = rotary_angles(64, 500000.0, kind, 8.0, original=8192)
        ratio = plain / f
        assert ratio[0] == 1.0 and ratio[-1].item() == pytest.approx(8.0, rel=1e-14), kind
        assert bool((ratio[1:] >= ratio[:-1] * (1 - 1e-14)).all()), kind
        assert bool(((ratio > 1.1) & (ratio < 7.9)).any()), kind        # a blend between the two ends
        assert scale == (1.0 if kind == "bands" else pytest.approx(0.1 * math.log(8.0) + 1))
        assert torch.allclose(rotary_angles(64, 500000.0, kind, 1.0)[0], plain, rtol=1e-14)
    assert rotary_angles(2)[0].tolist() == [1.0]


def test_rotary_plan_is_the_exact_fraction_of_a_turn():
    plan = ops.rotary_plan(8, inv_freq=torch.tensor([math.pi, 1.0, -0.5, 2 * math.pi], dtype=torch.float64),
                           layout="interleaved", scale=1.25, device="cpu")
    bits = [b % 2 ** 64 for b in plan.freq.tolist()]
    assert bits[0] == 2 ** 63 and bits[3] == 0      # half a turn; a whole turn is none
    assert bits[1] / 2 ** 64 == pytest.approx(1 / (2 * math.pi), rel=1e-15)
    assert (bits[2] + round(0.25 / math.pi * 2 ** 64)) % 2 ** 64 == 0
    assert plan.scale == 1.25 and plan.layout == L.LORA_ROTARY_INTERLEAVED and plan.rot_dim == 8


@pytest.mark.parametrize("kw", [dict(rot_dim=7), dict(rot_dim=0), dict(layout="other"), dict(scaling="other"),
                                dict(base=1.0), dict(scaling="linear", factor=0.5), dict(scale=float("inf")),
                                dict(scaling="bands", low=4.0, high=4.0), dict(inv_freq=torch.ones(3)),
                                dict(inv_freq=torch.tensor([1.0, 1.0, 1.0, float("nan")])),
                                dict(inv_freq=torch.ones(4), scaling="linear"), dict(inv_freq=torch.ones(4), factor=2.0)])
def test_rotary_plan_refusals(kw):
    with pytest.raises(ValueError):
        ops.rotary_plan(**{"rot_dim": 8, "device": "cpu", **kw})


# ------------------------------------------------------------------ refusals of the wrappers
def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


@pytest.mark.parametrize("kw", [
    dict(Y=_t(8, 24)), dict(Y=_t(7, 32)), dict(Y=_t(8, 32, dtype=torch.float32)), dict(Y=_t(32, 8).t()),
    dict(Y=_t(1, 32).expand(8, 32)), dict(w_pre=_t(24)), dict(w_pre=_t(32, dtype=torch.float32)),
    dict(w_post=_t(32)), dict(Y=None, post_norm=True), dict(Y=None, gate=_t(8, 32)), dict(Y=None, pre_norm=False),
    dict(w_pre=_t(32), pre_norm=False), dict(gate=_t(3, 32)), dict(gate=_t(4, 24)), dict(gate=_t(32)),
    dict(gate=_t(4, 32), rows_per_gate=3), dict(gate=_t(0, 32)), dict(X=_t(8)), dict(X=_t(8, 32).half()), dict(),
])
def test_norm_forward_refusals(kw):
    """The last case is well formed but for the device: CPU tensors never reach a kernel."""
    a = {"X": _t(8, 32), "Y": _t(8, 32), **kw}
    with pytest.raises((ValueError, TypeError)):
        ops.block_norm_fwd(**a)


@pytest.mark.parametrize("kw", [
    dict(dH=None, dXout=None), dict(dH=_t(8, 24)), dict(dXout=_t(7, 32)), dict(r_pre=None), dict(r_post=None),
    dict(r_pre=_t(7, dtype=torch.float32)), dict(r_pre=_t(8)), dict(Y=None), dict(w_post=_t(24)),
    dict(gate=_t(3, 32)), dict(),
])
def test_norm_backward_refusals(kw):
    f = torch.float32
    a = {"Xout": _t(8, 32), "Y": _t(8, 32), "r_pre": _t(8, dtype=f), "r_post": _t(8, dtype=f), "dH": _t(8, 32),
         "dXout": _t(8, 32), "post_norm": True, **kw}
    with pytest.raises((ValueError, TypeError)):
        ops.block_norm_bwd(**a)


@pytest.mark.parametrize("kw", [
    dict(X=_t(6, 32)), dict(X=_t(6, 2, 32).transpose(1, 2)), dict(X=_t(6, 2, 6)), dict(X=_t(6, 2, 32).half()),
    dict(pos=torch.arange(5)), dict(pos=torch.arange(6).float()), dict(pos=torch.arange(12)[::2]),
    dict(out=_t(6, 2, 24)), dict(out=_t(6, 2, 32, dtype=torch.float32)), dict(),
])
def test_rotary_refusals(kw):
    plan = ops.rotary_plan(8, device="cpu")
    a = {"X": _t(6, 2, 32), "pos": torch.arange(6), "out": None, **kw}
    for call in (ops.rotary_fwd, ops.rotary_bwd):
        with pytest.raises((ValueError, TypeError)):
            call(a["X"], a["pos"], plan, out=a["out"])


@pytest.mark.parametrize("kw", [dict(), dict(params=[]), dict(params=[_t(4).half()])])
def test_adamw_refuses_cpu_and_other_tensors(kw):
    with pytest.raises(ValueError):
        optim.AdamW(**{"params": [_t(4, 4)], **kw})


# ------------------------------------------------------------------ refusals of the C ABI
FAKE = ctypes.c_void_p(1 << 20)        # never dereferenced: the checks come first
ODD = ctypes.c_void_p((1 << 20) + 2)
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


def _norm_shape(**kw):
    a = dict(M=64, D=256, rows_per_gate=1, ldx=256, ldy=256, lddh=256, lddz=256, alpha=1.0, eps=1e-6, w_offset=0.0,
             post_norm=0, dtype=L.LORA_BF16)
    a.update(kw)
    return L.LoraNormShape(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(D=0), INVALID), (dict(D=252), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(alpha=float("inf")), INVALID),
    (dict(w_offset=float("nan")), INVALID), (dict(ldx=248), INVALID), (dict(ldy=260), MISALIGNED),
    (dict(M=1 << 31), UNSUPPORTED), (dict(rows_per_gate=-1), INVALID),
])
def test_norm_abi_shapes(lib, kw, status):
    sh = _norm_shape(**kw)
    args = [FAKE] * 2 + [None] * 3 + [FAKE] * 2 + [None] * 2
    assert lib.block_norm_fwd(ctypes.byref(sh), *args, None) == status
    assert L.block_norm_bwd_workspace_bytes(sh) == 0
    assert lib.block_norm_bwd(ctypes.byref(sh), FAKE, None, None, None, None, FAKE, None, FAKE, None, FAKE, None, None,
                              None, None, FAKE, 1 << 30, None) == status


def test_norm_abi_arguments(lib):
    names = ("X", "Y", "w_pre", "w_post", "gate", "Xout", "H", "r_pre", "r_post")
    out = ctypes.c_void_p(2 << 20)

    def fwd(sh=None, **kw):
        a = dict(X=FAKE, Y=FAKE, w_pre=None, w_post=None, gate=None, Xout=out, H=out, r_pre=None, r_post=None)
        a.update(kw)
        return lib.block_norm_fwd(ctypes.byref(sh or _norm_shape()), *[a[n] for n in names], None)

    assert lib.block_norm_fwd(None, *[FAKE] * 9, None) == INVALID
    assert fwd(X=None) == INVALID and fwd(Xout=None) == INVALID
    assert fwd(w_post=FAKE) == INVALID                                  # a weight without its norm
    assert fwd(w_pre=FAKE, H=None) == INVALID
    assert fwd(Y=None) == INVALID                                       # Xout without a block output
    assert fwd(Y=None, Xout=None, gate=FAKE) == INVALID
    assert fwd(Y=None, Xout=None, H=None) == INVALID
    assert fwd(_norm_shape(post_norm=1), Y=None, Xout=None) == INVALID
    assert fwd(_norm_shape(rows_per_gate=0), gate=FAKE) == INVALID
    assert fwd(_norm_shape(ldx=264), Xout=FAKE) == INVALID              # in place with another row stride
    for n in names:
        a = dict(w_pre=FAKE, w_post=FAKE, gate=FAKE, r_pre=FAKE, r_post=FAKE)
        a[n] = ODD
        assert fwd(_norm_shape(post_norm=1), **a) == MISALIGNED, n
    assert fwd(_norm_shape(M=0)) == 0                                   # no rows: nothing to do

    bnames = ("Xout", "Y", "w_pre", "w_post", "gate", "r_pre", "r_post", "dH", "dXout", "dX", "dY", "dw_pre", "dw_post",
              "dgate")

    def bwd(sh=None, ws=FAKE, size=1 << 30, **kw):
        a = dict.fromkeys(bnames, FAKE)
        a.update(dict(dX=out, dY=out, dw_pre=out, dw_post=out, dgate=out))
        a.update(kw)
        return lib.block_norm_bwd(ctypes.byref(sh or _norm_shape(post_norm=1)), *[a[n] for n in bnames], ws, size, None)

    assert bwd(Xout=None) == INVALID and bwd(dH=None, dXout=None) == INVALID
    assert bwd(r_pre=None) == INVALID and bwd(r_post=None) == INVALID
    assert bwd(Y=None) == INVALID and bwd(_norm_shape()) == INVALID     # w_post without its norm
    assert bwd(w_pre=None) == INVALID and bwd(w_post=None) == INVALID and bwd(gate=None) == INVALID
    assert bwd(dX=FAKE) == INVALID and bwd(dY=FAKE) == INVALID          # an output on an input
    assert bwd(_norm_shape(post_norm=1, rows_per_gate=0)) == INVALID
    for n in bnames:
        assert bwd(**{n: ODD}) == MISALIGNED, n
    assert bwd(ws=None) == WORKSPACE and bwd(size=256) == WORKSPACE
    assert bwd(ws=ctypes.c_void_p((1 << 20) + 16)) == MISALIGNED
    assert L.block_norm_bwd_workspace_bytes(_norm_shape()) >= 256 + 64 * 4


def _rot_shape(**kw):
    a = dict(M=8, H=4, head_dim=64, rot_dim=64, x_token=256, x_head=64, y_token=256, y_head=64, scale=1.0, layout=0,
             pos_bits=64, dtype=L.LORA_BF16)
    a.update(kw)
    return L.LoraRotaryShape(**a)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), INVALID), (dict(H=0), INVALID), (dict(rot_dim=63), INVALID), (dict(rot_dim=0), INVALID),
    (dict(rot_dim=66), INVALID), (dict(layout=2), INVALID), (dict(pos_bits=16), INVALID), (dict(dtype=5), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(M=1 << 31), UNSUPPORTED), (dict(head_dim=4098, rot_dim=8), UNSUPPORTED),
    (dict(y_head=32), INVALID), (dict(y_token=128), INVALID), (dict(y_token=0), INVALID), (dict(x_token=-256), INVALID),
    (dict(y_token=64, y_head=64), INVALID),
])
def test_rotary_abi_shapes(lib, kw, status):
    for call in (lib.rotary_fwd, lib.rotary_bwd):
        assert call(ctypes.byref(_rot_shape(**kw)), FAKE, FAKE, FAKE, ctypes.c_void_p(2 << 20), None) == status


def test_rotary_abi_arguments(lib):
    out = ctypes.c_void_p(2 << 20)
    ok = ctypes.byref(_rot_shape())
    assert lib.rotary_fwd(None, FAKE, FAKE, FAKE, out, None) == INVALID
    for args in ((None, FAKE, FAKE, out), (FAKE, None, FAKE, out), (FAKE, FAKE, None, out), (FAKE, FAKE, FAKE, None)):
        assert lib.rotary_fwd(ok, *args, None) == INVALID
    one = ctypes.c_void_p((1 << 20) + 1)
    for args in ((one, FAKE, FAKE, out), (FAKE, ODD, FAKE, out), (FAKE, FAKE, ODD, out), (FAKE, FAKE, FAKE, one)):
        assert lib.rotary_fwd(ok, *args, None) == MISALIGNED
    assert lib.rotary_fwd(ctypes.byref(_rot_shape(dtype=L.LORA_F32)), ODD, FAKE, FAKE, out, None) == MISALIGNED
    assert lib.rotary_fwd(ctypes.byref(_rot_shape(x_token=512)), FAKE, FAKE, FAKE, FAKE, None) == INVALID  # in place
    assert lib.rotary_fwd(ctypes.byref(_rot_shape(M=0)), None, None, FAKE, None, None) == 0


def _adamw_args(n=1000, dtype=L.LORA_BF16, p=1 << 20, g=1 << 20, lr_mul=1.0, decay=0.0):
    return (L.LoraAdamwTensor * 1)(L.LoraAdamwTensor(p, n, lr_mul, decay, dtype)), (ctypes.c_void_p * 1)(g)


def _adamw_state(**kw):
    a = dict(m=1 << 20, v=1 << 20, m_scale=1 << 20, v_scale=1 << 20, master=1 << 20, ctl=1 << 20, bits=32)
    a.update(kw)
    return L.LoraAdamwState(**a)


def _hyper(**kw):
    a = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, grad_scale=1.0, lr_device=None)
    a.update(kw)
    return L.LoraAdamwHyper(**a)


def test_adamw_abi(lib):
    t, g = _adamw_args()
    two = (L.LoraAdamwTensor * 2)(L.LoraAdamwTensor(1 << 20, 257, 1.0, 0.0, 0), L.LoraAdamwTensor(None, 0, 1.0, 0.0, 0))
    assert L.adamw_state_blocks(t, 1) == 4 and L.adamw_state_blocks(two, 2) == 2 and L.adamw_state_blocks(two, -1) == -1
    assert L.adamw_norm_workspace_bytes(-1) == 0 and L.adamw_norm_workspace_bytes(0) > 256

    def step(t=t, g=g, count=1, state=None, hyper=None, coef=None):
        s, h = state or _adamw_state(), hyper or _hyper()
        return lib.adamw_step(t, g, count, ctypes.byref(s), ctypes.byref(h), coef, None)

    assert step(count=-1) == INVALID and step(t=None) == INVALID and step(g=None) == INVALID
    for bad, status in ((dict(n=-1), INVALID), (dict(dtype=7), INVALID), (dict(p=None), INVALID),
                        (dict(p=(1 << 20) + 1), MISALIGNED), (dict(g=(1 << 20) + 1), MISALIGNED),
                        (dict(lr_mul=float("nan")), INVALID), (dict(decay=float("inf")), INVALID),
                        (dict(n=1 << 40), UNSUPPORTED)):
        tb, gb = _adamw_args(**bad)
        assert step(t=tb, g=gb) == status, bad
        assert lib.adamw_grad_norm(tb, gb, 1, 1.0, 1.0, FAKE, FAKE, 1 << 30, None) == status, bad
    for bad, status in ((dict(bits=16), INVALID), (dict(ctl=None), INVALID), (dict(m=None), INVALID),
                        (dict(v=None), INVALID), (dict(m=(1 << 20) + 8), MISALIGNED),
                        (dict(master=(1 << 20) + 4), MISALIGNED), (dict(ctl=(1 << 20) + 4), MISALIGNED),
                        (dict(bits=8, m_scale=None), INVALID), (dict(bits=8, v_scale=None), INVALID)):
        assert step(state=_adamw_state(**bad)) == status, bad
    for bad in (dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=float("nan")), dict(eps=0.0), dict(eps=float("inf")),
                dict(lr=float("nan")), dict(grad_scale=float("inf"))):
        assert step(hyper=_hyper(**bad)) == INVALID, bad
    assert step(hyper=_hyper(lr_device=(1 << 20) + 2)) == MISALIGNED and step(coef=ODD) == MISALIGNED
    none = (ctypes.c_void_p * 1)(None)
    assert step(g=none) == 0 and step(count=0) == 0       # nothing has a gradient: nothing is launched

    fill = lambda t=t, n=1, to=FAKE: lib.adamw_fill_master(t, n, to, None)  # noqa: E731
    assert fill(t=None) == INVALID and fill(n=-1) == INVALID and fill(to=None) == INVALID and fill(to=ODD) == MISALIGNED
    assert fill(t=_adamw_args(p=None)[0]) == INVALID and fill(t=_adamw_args(p=(1 << 20) + 1)[0]) == MISALIGNED
    assert fill(n=0, to=None) == 0

    def norm(coef=FAKE, scale=1.0, most=1.0, ws=FAKE, size=1 << 30):
        return lib.adamw_grad_norm(t, g, 1, scale, most, coef, ws, size, None)

    assert norm(coef=None) == INVALID and norm(scale=float("nan")) == INVALID and norm(most=float("nan")) == INVALID
    assert norm(coef=ctypes.c_void_p((1 << 20) + 4)) == MISALIGNED
    assert norm(ws=None) == WORKSPACE and norm(size=256) == WORKSPACE
