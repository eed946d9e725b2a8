"""The many-adapter projection without a GPU: its fp64 reference against differences and against the
one-adapter layer's, and every refusal."""
import ctypes

import numpy as np
import pytest
import torch

import oracle as O1
from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import adapters, ops, optim
from oracle import multi_oracle as O


def _case(seed=0, M=7, d_in=6, d_out=5, r=3, n=3):
    g = np.random.default_rng(seed)
    return (g.normal(size=(M, d_in)), g.normal(size=(d_out, d_in)), g.normal(size=(n, r, d_in)),
            g.normal(size=(n, d_out, r)), g.normal(size=n), np.array([0, 2, -1, 2, 5, 0, 2]))


def test_reference_is_the_one_adapter_layer_on_its_rows():
    X, W0, A, B, s, ids = _case()
    Y, Z = O.multi_fwd(X, W0, A, B, s, ids, bias=np.arange(5.0))
    dY = np.random.default_rng(1).normal(size=Y.shape)
    dX, dA, dB, db, _ = O.multi_bwd(X, W0, A, B, s, ids, Z, dY)
    for a in range(3):
        at = ids == a
        np.testing.assert_allclose(Y[at], O1.lora_linear_fwd(X[at], W0, A[a], B[a], s[a]) + np.arange(5.0), rtol=1e-12)
        rX, rA, rB, _ = O1.lora_linear_bwd(X[at], W0, A[a], B[a], s[a], dY[at])
        for got, ref in ((dX[at], rX), (dA[a], rA), (dB[a], rB)):
            np.testing.assert_allclose(got, ref, rtol=1e-10, atol=1e-12)
    bare = (ids < 0) | (ids > 2)
    np.testing.assert_allclose(Y[bare], X[bare] @ W0.T + np.arange(5.0))
    np.testing.assert_allclose(dX[bare], dY[bare] @ W0)
    assert not dA[1].any() and not dB[1].any() and not Z[bare].any()
    np.testing.assert_allclose(db, dY.sum(0))


def test_reference_gradients_are_differences():
    X, W0, A, B, s, ids = _case(2)
    dY = np.random.default_rng(3).normal(size=(7, 5))
    Z = O.multi_fwd(X, W0, A, B, s, ids)[1]
    grads = O.multi_bwd(X, W0, A, B, s, ids, Z, dY)
    loss = lambda: float((O.multi_fwd(X, W0, A, B, s, ids)[0] * dY).sum())  # noqa: E731
    for t, g in ((X, grads[0]), (A, grads[1]), (B, grads[2])):
        for at in [tuple(np.random.default_rng(4 + k).integers(0, t.shape)) for k in range(12)]:
            keep, h = t[at], 1e-5
            t[at] = keep + h
            up = loss()
            t[at] = keep - h
            down = loss()
            t[at] = keep
            assert abs((up - down) / (2 * h) - g[at]) < 1e-7 * max(1.0, abs(g[at]))


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def _ok():
    plan = adapters.AdapterPlan(8, 3, "cpu")
    return dict(X=_t(8, 32), W0=_t(16, 32), A=_t(3, 8, 32), B=_t(3, 16, 8), s=1.0, plan=plan)


@pytest.mark.parametrize("name,bad", [
    ("X", _t(8, 40)), ("X", _t(9, 32)), ("X", _t(8, 2, 16)), ("X", _t(8, 64)[:, ::2]),
    ("W0", _t(16, 40)), ("W0", _t(32, 16).t()), ("W0", _t(16, 32, dtype=torch.float32)),
    ("A", _t(8, 32)), ("A", _t(3, 8, 40)), ("A", _t(2, 8, 32)), ("A", _t(3, 32, 8).transpose(1, 2)),
    ("B", _t(3, 16, 16)), ("B", _t(3, 24, 8)), ("B", _t(4, 16, 8)), ("B", _t(3, 8, 16).transpose(1, 2)),
    ("s", float("nan")), ("s", float("inf")), ("s", _t(3)), ("s", torch.zeros(4)), ("s", torch.zeros(6)[::2]),
    ("plan", None), ("plan", adapters.AdapterPlan(9, 3, "cpu")), ("plan", adapters.AdapterPlan(8, 4, "cpu")),
    ("bias", _t(15)), ("bias", _t(16, dtype=torch.float32)),
])
def test_forward_refuses(name, bad):
    a = dict(_ok(), **{name: bad})
    with pytest.raises(ValueError):
        ops.lora_multi_fwd(**a)


@pytest.mark.parametrize("name,bad", [("Z", _t(8, 16)), ("Z", _t(7, 8)), ("Z", _t(8, 8, dtype=torch.float32)),
                                      ("dY", _t(8, 24)), ("dY", _t(16, 8).t()), ("dY", None), ("A", _t(3, 8, 40)),
                                      ("plan", adapters.AdapterPlan(8, 2, "cpu"))])
def test_backward_refuses(name, bad):
    a = dict(_ok(), Z=_t(8, 8), dY=_t(8, 16))
    a[name] = bad
    with pytest.raises(ValueError):
        ops.lora_multi_bwd(**a)


def test_cpu_tensors_are_refused():
    with pytest.raises(ValueError, match="CUDA"):
        ops.lora_multi_fwd(**_ok())
    with pytest.raises(ValueError, match="CUDA"):
        ops.lora_multi_bwd(**_ok(), Z=None, dY=_t(8, 16))


@pytest.mark.parametrize("s", [1e39, -1e300, 2 ** 200])
def test_a_scale_beyond_fp32_is_refused(s):
    with pytest.raises(ValueError, match="s must be finite"):
        ops.lora_multi_fwd(**dict(_ok(), s=s))


@pytest.mark.parametrize("ids", [torch.zeros(4), torch.zeros(2, 2, dtype=torch.int64),
                                 torch.zeros(8, dtype=torch.int64)[::2], torch.zeros(4, dtype=torch.int16),
                                 torch.zeros(4, dtype=torch.int64)])
def test_plan_refuses_ids(ids):
    with pytest.raises(ValueError):
        ops.adapter_plan(ids, 3)


@pytest.mark.parametrize("rows,n", [(-1, 3), (2 ** 24 + 1, 3), (4, 0), (4, 65536), (4, -2)])
def test_plan_refuses_sizes(rows, n):
    assert L.lora_multi_plan_bytes(rows, n) == 0
    with pytest.raises(ValueError):
        adapters.AdapterPlan(rows, n, "cpu")


def test_plan_update_keeps_its_size():
    plan = adapters.AdapterPlan(4, 3, "cpu")
    with pytest.raises(ValueError):
        plan.update(torch.zeros(5, dtype=torch.int64))


def test_entry_points_check_before_they_launch():
    lib = L._lib()
    fake, odd = ctypes.c_void_p(1 << 20), ctypes.c_void_p((1 << 20) + 4)
    big = 1 << 40
    shape = lambda *a: L.LoraMultiShape(*a)  # noqa: E731

    def fwd(sh, X=fake, W0=fake, A=fake, B=fake, bias=None, s=1.0, each=None, plan=fake, Y=fake, Z=None, ws=fake, n=big):
        return lib.lora_multi_fwd(ctypes.byref(sh) if sh else None, X, W0, A, B, bias, s, each, plan, Y, Z, ws, n, None)

    def bwd(sh, X=fake, A=fake, Z=None, dY=fake, s=1.0, plan=fake, dX=None, dA=fake, dB=fake, ws=fake, n=big):
        return lib.lora_multi_bwd(ctypes.byref(sh), X, fake, A, fake, Z, dY, s, None, plan, dX, dA, dB, None, ws, n, None)

    ok = shape(64, 256, 128, 8, 4, L.LORA_BF16)
    need = L.lora_multi_workspace_bytes(False, ok), L.lora_multi_workspace_bytes(True, ok)
    assert min(need) > 256
    for call in (fwd, bwd):
        assert call(ok, X=None) == 1 and call(ok, A=None) == 1 and call(ok, plan=None) == 1
        assert call(ok, X=odd) == 3 and call(ok, plan=odd) == 3
        assert call(ok, s=float("nan")) == 1
        assert call(ok, ws=None) == 4 and call(ok, n=need[call is bwd] - 1) == 4
    assert fwd(None) == 1 and fwd(ok, Y=None) == 1 and fwd(ok, Z=odd) == 3 and fwd(ok, bias=odd) == 3
    assert fwd(ok, each=ctypes.c_void_p((1 << 20) + 2)) == 3
    assert bwd(ok, dY=None) == 1 and bwd(ok, dA=None) == 1 and bwd(ok, dB=odd) == 3 and bwd(ok, dX=odd) == 3
    for bad, status in ((shape(-1, 256, 128, 8, 4, 1), 1), (shape(64, 0, 128, 8, 4, 1), 1), (shape(64, 256, 0, 8, 4, 1), 1),
                        (shape(64, 256, 128, 0, 4, 1), 1), (shape(64, 256, 128, 8, 0, 1), 1), (shape(64, 256, 128, 8, 4, 2), 1),
                        (shape(64, 252, 128, 8, 4, 1), 2), (shape(64, 256, 124, 8, 4, 1), 2),
                        (shape(64, 256, 128, 12, 4, 1), 2), (shape(64, 256, 128, 136, 4, 1), 2),
                        (shape(64, 256, 128, 129, 4, 0), 2), (shape(2 ** 24 + 1, 256, 128, 8, 4, 1), 2),
                        (shape(64, 256, 128, 8, 65536, 1), 2), (shape(64, 2 ** 31, 128, 8, 4, 1), 2)):
        assert fwd(bad) == status and bwd(bad) == status, (bad.M, bad.d_in, bad.d_out, bad.r, bad.n, bad.dtype)
        assert L.lora_multi_workspace_bytes(False, bad) == 0 == L.lora_multi_workspace_bytes(True, bad)
    assert L.lora_multi_workspace_bytes(False, shape(64, 256, 128, 13, 4, L.LORA_F32)) > 0
    none = shape(0, 256, 128, 8, 4, 1)
    assert fwd(none, X=None, Y=None) == 0       # no rows: nothing to do
    plan = lambda M=4, n=3, ids=fake, bits=64, p=fake, size=big: lib.lora_multi_plan(M, n, ids, bits, p, size, None)  # noqa: E731
    assert plan(M=-1) == 1 and plan(n=0) == 1 and plan(n=65536) == 2 and plan(M=2 ** 24 + 1) == 2
    assert plan(ids=None) == 1 and plan(bits=16) == 1 and plan(ids=odd) == 3 and plan(p=None) == 4
    assert plan(p=odd) == 3 and plan(size=L.lora_multi_plan_bytes(4, 3) - 1) == 4 and plan(M=0, ids=None) == 0


# ------------------------------------------------------------------ clipping by groups
def test_clip_reference():
    g = np.random.default_rng(0)
    grads = [g.normal(size=(3, 4)) * 10, g.normal(size=5) * 0.01, g.normal(size=2) * 10]
    norms, out = O.clip(grads, 1.0, [0, 1, 0], 3)
    t = [torch.nn.Parameter(torch.zeros(v.shape)) for v in (grads[0], grads[2])]
    for p, v in zip(t, (grads[0], grads[2])):
        p.grad = torch.from_numpy(v.copy()).float()
    total = torch.nn.utils.clip_grad_norm_(t, 1.0)
    assert abs(norms[0] - float(total)) < 1e-5 * norms[0] and norms[2] == 0
    np.testing.assert_allclose(out[0], t[0].grad.numpy(), rtol=1e-5)
    np.testing.assert_allclose(out[2], t[1].grad.numpy(), rtol=1e-5)
    assert (out[1] == grads[1]).all()
    grads[1][0] = np.inf
    norms, out = O.clip(grads, 1.0, [0, 1, 0], 3)
    assert not out[1].any() and np.isinf(norms[1]) and abs(np.sqrt((out[0] ** 2).sum() + (out[2] ** 2).sum()) - 1) < 1e-6


@pytest.mark.parametrize("kw,what", [
    (dict(grads=[torch.zeros(4)], max_norm=1.0), "CUDA"),
    (dict(grads=[3.0], max_norm=1.0), "tensor or None"),
    (dict(grads=[], max_norm=1.0), "no gradients"),
    (dict(grads=[None], max_norm=1.0), "no gradients"),
    (dict(grads=[torch.zeros(4)], max_norm=0.0), "max_norm"),
    (dict(grads=[torch.zeros(4)], max_norm=-1.0), "max_norm"),
    (dict(grads=[torch.zeros(4)], max_norm=float("nan")), "max_norm"),
    (dict(grads=[torch.zeros(4)], max_norm=1e-60), "max_norm"),
    (dict(grads=[torch.zeros(4)], max_norm=1.0, groups=[0, 1]), "2 groups"),
    (dict(grads=[torch.zeros(4)], max_norm=1.0, groups=0), "1 to 65535"),
    (dict(grads=[torch.zeros(4)], max_norm=1.0, groups=70000), "1 to 65535"),
    (dict(grads=[None, None], max_norm=1.0, groups=[0, 70000]), "1 to 65535"),
])
def test_clip_refuses(kw, what):
    with pytest.raises(ValueError, match=what):
        optim.clip_grads(**kw)


def test_clip_entry_point_checks_before_it_launches():
    lib = L._lib()
    p = ctypes.c_void_p(1 << 20)

    def call(*tensors, groups=2, stacked=0, max_norm=1.0, norms=p, ws=p, size=1 << 30, count=None):
        t = (L.LoraGradTensor * max(len(tensors), 1))(*tensors)
        return lib.grad_clip(t, len(tensors) if count is None else count, groups, stacked, max_norm, norms, ws, size, None)

    a, b = (1 << 20, 100, 0, 0), (1 << 21, 64, 1, 1)
    assert call(a, groups=0) == 1 and call(a, groups=65536) == 2 and call(a, count=-1) == 1
    assert call((1 << 20, -1, 0, 0)) == 1 and call((None, 4, 0, 0)) == 1 and call((1 << 20, 4, 0, 2)) == 1
    assert call((1 << 20, 4, 2, 0)) == 1 and call((1 << 20, 4, -1, 0)) == 1       # the group
    assert call(((1 << 20) + 2, 4, 0, 0)) == 3 and call(((1 << 20) + 1, 4, 0, 1)) == 3
    assert call(a, a) == 1 and call(a, b, ((1 << 20) + 396, 8, 1, 0)) == 1       # shared memory
    assert call(((1 << 21) - 384, 100, 0, 1), b, stacked=1) == 1       # 2 groups of 200 bytes
    assert call(a, b, norms=None) == 1 and call(a, b, norms=ctypes.c_void_p(2)) == 3 and call(a, b, max_norm=float("nan")) == 1
    t = (L.LoraGradTensor * 2)(a, b)
    need = L.grad_clip_workspace_bytes(t, 2, 2, False)
    assert need > 0 and call(a, b, size=need - 1) == 4 and call(a, b, ws=None) == 4
    assert call(a, b, ws=ctypes.c_void_p((1 << 20) + 8)) == 3
    assert L.grad_clip_workspace_bytes(t, 2, 0, False) == 0
    assert call((1 << 20, 2 ** 46, 0, 0)) == 2                          # more units than are counted
