"""Block norm, rotary positions and AdamW on the GPU against the fp64 reference.

Every element is held to a bound made of the one rounding of its store, u |ref| (u = 2^-8 for bf16,
2^-24 for fp32), and of k fp32 roundings (2^-24 each) of the magnitudes that the formula adds: the
reference's own formula over absolute values.  k counts the longest chain of fp32 operations (the
additions of a row sum are at most 64 deep, a column sum's at most M + 64)."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as BO
from parity import to64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E32 = 2.0 ** -24
UNIT = {dt: torch.finfo(dt).eps / 2 for dt in (torch.bfloat16, torch.float32)}      # half a spacing: 2^-8, 2^-24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def ops():
    from dora_adapter_linear_gb300.build import build
    build()
    from dora_adapter_linear_gb300 import ops as _ops
    return _ops


@pytest.fixture(scope="module")
def optim(ops):
    from dora_adapter_linear_gb300 import optim as _optim
    return _optim


def f64(t):
    return None if t is None else to64(t)


def within(got, ref, slack, dtype, what):
    """|got - ref| <= 1.01 u |ref| + slack, element by element."""
    got = to64(got)
    assert got.shape == ref.shape and np.isfinite(got).all(), what
    over = np.abs(got - ref) - (1.01 * UNIT[dtype] * np.abs(ref) + slack)
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over the bound at {np.unravel_index(over.argmax(), over.shape)}"


# ------------------------------------------------------------------ block norm
def norm_case(M, D, dtype, gate, post, y=True, pre=True, off=0.0, alpha=1.0, seed=0, rpg=None):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s, scale=1.0, mean=0.0: (torch.randn(*s, generator=gen) * scale + mean).to(dtype).to(DEV)  # noqa: E731
    rpg = {"none": None, "row": max(M, 1), "token": 1}.get(gate, rpg)
    t = dict(X=n(M, D, scale=2.0), Y=n(M, D) if y else None, dH=n(M, D) if pre else None, dXout=n(M, D))
    kw = dict(w_pre=n(D, scale=0.3, mean=1 - off) if pre else None, w_post=n(D, scale=0.3, mean=1 - off) if post else None,
              gate=n(-(-M // rpg), D) if rpg else None, rows_per_gate=rpg, alpha=alpha, w_offset=off, post_norm=post)
    return t, kw


def ref_kw(kw):
    return dict(w_pre=f64(kw["w_pre"]), w_post=f64(kw["w_post"]), gate=f64(kw["gate"]),
                rows_per_gate=kw["rows_per_gate"] or 1, alpha=float(np.float32(kw["alpha"])),
                off=float(np.float32(kw["w_offset"])), post=kw["post_norm"])


def check_norm_fwd(got, t, kw, pre, dtype, eps):
    k = ref_kw(kw)
    x, y, eps = f64(t["X"]), f64(t["Y"]), float(np.float32(eps))
    z, h, r_pre, r_post = BO.block_norm_fwd(x, y, eps=eps, **k)
    mag = np.abs(x)
    if y is not None:
        mag = mag + np.abs(z - x)
        within(got[0], z, 72 * E32 * mag, dtype, "Xout")
        if k["post"]:
            assert np.allclose(to64(got[3]), r_post, rtol=64 * E32, atol=0)
    if not pre:
        assert got[1] is None and got[2] is None
        return
    rho = (np.abs(z) * mag).sum(1, keepdims=True) / np.maximum((z ** 2).sum(1, keepdims=True), 1e-300)
    rel = 72 * rho + 72
    r, w = r_pre[:, None], 1.0 if k["w_pre"] is None else k["w_pre"] + k["off"]
    within(got[1], h, E32 * (72 * np.abs(w * r) * mag + rel * np.abs(h)), dtype, "H")
    assert (np.abs(to64(got[2]) - r_pre) <= E32 * rel[:, 0] * r_pre).all()


def check_norm_bwd(got, Xout, t, kw, r_pre, r_post, dtype):
    k = ref_kw(kw)
    z, y, dh, dzi = f64(Xout), f64(t["Y"]), f64(t["dH"]), f64(t["dXout"])
    r_pre, r_post = f64(r_pre), f64(r_post)
    ref = BO.block_norm_bwd(z, y, r_pre, r_post, dh, dzi, **k)
    M, D = z.shape
    a = np.abs
    mag = np.zeros((M, D)) if dzi is None else a(dzi)
    c = np.zeros((M, 1))
    if dh is not None:
        rz, wdh = r_pre[:, None], a(dh * (1.0 if k["w_pre"] is None else k["w_pre"] + k["off"]))
        c = rz ** 3 / D * (wdh * a(z)).sum(1, keepdims=True)
        mag = mag + rz * wdh + c * a(z)
        within(got[2], ref[2], (M + 64) * E32 * a(dh * z * rz).sum(0), dtype, "dw_pre") if k["w_pre"] is not None else None
    within(got[0], ref[0], 96 * E32 * mag, dtype, "dX")
    if y is None:
        assert got[1] is None and got[3] is None and got[4] is None
        return
    g = a(k["alpha"] * BO._rows(k["gate"], M, k["rows_per_gate"]))
    dp, p = g * mag, a(y)
    dy, w = dp, 1.0
    if k["post"]:
        w, n = (1.0 if k["w_post"] is None else a(k["w_post"] + k["off"])), a(y) * r_post[:, None]
        p = n * w
        dy = r_post[:, None] * (w * dp + n * (w * dp * n).mean(1, keepdims=True))
        if k["w_post"] is not None:
            within(got[3], ref[3], (M + 128) * E32 * (dp * n).sum(0), dtype, "dw_post")
    within(got[1], ref[1], 128 * E32 * dy, dtype, "dY")
    if k["gate"] is not None:
        s = np.zeros_like(k["gate"])
        np.add.at(s, np.arange(M) // k["rows_per_gate"], a(k["alpha"]) * mag * p)
        within(got[4], ref[4], (k["rows_per_gate"] + 128) * E32 * s, dtype, "dgate")


NORM_CASES = [  # M, D, gate, post, kwargs
    (1, 8, "none", True, {}), (1, 4096, "none", True, dict(off=1.0)), (1, 14336, "token", True, {}),
    (3, 40, "row", False, dict(alpha=0.22)), (77, 264, "token", True, dict(off=1.0)), (33, 1032, "seq", True, dict(rpg=7)),
    (129, 2568, "seq", False, dict(rpg=2)), (300, 768, "seq", True, dict(rpg=75, alpha=-0.5)),
    (1031, 512, "row", True, {}), (640, 1536, "none", True, dict(pre=False)), (200, 4096, "seq", True, dict(rpg=300)),
    (65, 8200, "row", True, {}), (40, 11008, "none", False, {}), (21, 20488, "seq", True, dict(rpg=10)),
    (90, 1024, "none", False, dict(y=False)), (5, 5120, "none", False, dict(y=False, off=1.0)),
    # enough rows that each variant walks, holds two vectors a thread, or takes two rows a barrier
    (1100, 2048, "none", True, dict(off=1.0)), (1300, 1544, "token", True, {}), (1250, 2048, "seq", True, dict(rpg=101)),
    (1500, 1032, "seq", False, dict(rpg=3)), (700, 4096, "row", False, {}), (2500, 520, "token", True, {}),
    (310, 8192, "seq", True, dict(rpg=4)), (400, 6008, "token", False, {}), (170, 16384, "none", True, {}),
    (350, 4104, "none", False, dict(y=False)), (3000, 400, "row", False, {}), (900, 504, "row", True, {}),
    (700, 128, "seq", True, dict(rpg=1)), (2000, 64, "seq", True, dict(rpg=3)), (9, 33000, "row", True, {}),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D,gate,post,more", NORM_CASES)
def test_norm(ops, M, D, gate, post, more, dtype):
    t, kw = norm_case(M, D, dtype, gate, post, seed=M + D, **more)
    pre = more.get("pre", True)
    got = ops.block_norm_fwd(t["X"], t["Y"], pre_norm=pre, eps=1e-5, **kw)
    check_norm_fwd(got, t, kw, pre, dtype, 1e-5)
    Xout, _, r_pre, r_post = got
    if t["Y"] is None:
        assert Xout is t["X"]
    grads = ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw)
    check_norm_bwd(grads, Xout, t, kw, r_pre, r_post, dtype)
    again = ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw)
    for a, b in zip(grads, again):
        assert (a is None and b is None) or torch.equal(a, b)      # sums in a fixed order


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D,gate,post,more", [
    (1, 64, "token", True, {}), (3, 8, "row", True, {}), (7, 128, "none", False, {}), (2500, 72, "none", True, dict(off=1.0)),
    (2600, 136, "seq", True, dict(rpg=16)), (10001, 64, "seq", False, dict(rpg=17)), (9000, 128, "token", True, {}),
    (5003, 256, "token", False, dict(alpha=-0.3)), (4099, 264, "seq", True, dict(rpg=64)), (4100, 512, "row", True, {}),
    (2700, 512, "token", True, dict(off=1.0)), (3000, 504, "none", False, dict(y=False)), (640, 40, "seq", True, dict(rpg=5)),
    (33, 256, "seq", True, dict(rpg=32)), (20000, 16, "none", True, {}), (700, 96, "none", False, dict(y=False)),
    (2503, 1024, "token", True, {}), (1501, 648, "seq", True, dict(rpg=16)), (702, 1000, "row", False, {}),
    (3, 1024, "none", True, {}), (1300, 776, "token", False, dict(off=1.0)), (2100, 392, "seq", False, dict(rpg=301)),
])
def test_norm_backward_of_short_rows(ops, M, D, gate, post, more, dtype):
    test_norm(ops, M, D, gate, post, more, dtype)


@pytest.mark.parametrize("D", [64, 120, 256, 512, 1024])
@pytest.mark.parametrize("which", ["dH", "dXout", "dX", "dw", "dgate"])
@pytest.mark.parametrize("gate", ["token", "seq"])
def test_norm_backward_of_short_rows_in_part(ops, D, which, gate):
    t, kw = norm_case(333, D, BF16, gate, True, seed=23, rpg=100)
    Xout, _, r_pre, r_post = ops.block_norm_fwd(t["X"], t["Y"], **kw)
    full = ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw)
    if which in t:
        t[which] = None
        check_norm_bwd(ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw), Xout, t, kw, r_pre,
                       r_post, BF16)
        return
    got = ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], need_dx=which != "dX",
                             need_dw=which != "dw", need_dgate=which != "dgate", **kw)
    for name, a, b in zip(("dX", "dY", "dw", "dw", "dgate"), got, full):
        assert a is None if name == which else torch.equal(a, b)


def test_norm_backward_of_short_rows_past_32_bit_offsets(ops):
    M, D, ld = 3, 256, (1 << 30) + 8
    t, kw = norm_case(M, D, BF16, "none", True, seed=24)
    X = torch.empty(2 * ld + D, dtype=BF16, device=DEV).as_strided((M, D), (ld, 1))
    X.copy_(t["X"])
    _, _, r_pre, r_post = ops.block_norm_fwd(t["X"], t["Y"], **kw)
    a, b = (ops.block_norm_bwd(x, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw) for x in (X, t["X"]))
    assert all(torch.equal(a[i], b[i]) for i in range(4))


@pytest.mark.parametrize("which", ["dH", "dXout"])
def test_norm_backward_with_one_gradient(ops, which):
    t, kw = norm_case(50, 520, BF16, "row", True, seed=4)
    Xout, _, r_pre, r_post = ops.block_norm_fwd(t["X"], t["Y"], **kw)
    t[which] = None
    check_norm_bwd(ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw), Xout, t, kw, r_pre,
                   r_post, BF16)


def test_norm_backward_returns_what_is_asked_for(ops):
    t, kw = norm_case(50, 520, BF16, "seq", True, seed=5, rpg=20)
    Xout, _, r_pre, r_post = ops.block_norm_fwd(t["X"], t["Y"], **kw)
    full = ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw)
    for want in ((False, True, True), (True, False, True), (True, True, False), (False, False, False)):
        got = ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], need_dx=want[0], need_dw=want[1],
                                 need_dgate=want[2], **kw)
        for i, keep in enumerate((want[0], True, want[1], want[1], want[2])):
            assert torch.equal(got[i], full[i]) if keep else got[i] is None, (want, i)


def test_norm_takes_strided_rows_and_weightless_norms(ops):
    t, kw = norm_case(37, 264, BF16, "row", True, seed=6)
    wide = {k: torch.full((37, 264 + 8 * i), float("nan"), dtype=BF16, device=DEV) for i, k in enumerate(t, 1)}
    for k, w in wide.items():
        w[:, :264] = t[k]
    s = {k: w[:, :264] for k, w in wide.items()}
    kw.update(w_pre=None, w_post=None)
    got, ref = (ops.block_norm_fwd(a["X"], a["Y"], **kw) for a in (s, t))
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    check_norm_fwd(got, t, kw, True, BF16, 1e-6)
    zs = torch.full((37, 400), float("nan"), dtype=BF16, device=DEV)[:, 64:328]
    zs.copy_(got[0])
    a = ops.block_norm_bwd(zs, s["Y"], got[2], got[3], s["dH"], s["dXout"], **kw)
    b = ops.block_norm_bwd(got[0], t["Y"], got[2], got[3], t["dH"], t["dXout"], **kw)
    assert a[2] is None and a[3] is None and all(torch.equal(a[i], b[i]) for i in (0, 1, 4))
    check_norm_bwd(b, got[0], t, kw, got[2], got[3], BF16)


def test_norm_rows_past_32_bit_offsets(ops):
    """Row strides that carry the last row past 2^31 elements."""
    M, D, ld = 3, 1024, (1 << 30) + 8
    big = torch.empty(2 * ld + D, dtype=BF16, device=DEV)
    X = big.as_strided((M, D), (ld, 1))
    t, kw = norm_case(M, D, BF16, "none", True, seed=7)
    X.copy_(t["X"])
    assert all(torch.equal(a, b) for a, b in zip(ops.block_norm_fwd(X, t["Y"], **{k: v for k, v in kw.items()}),
                                                 ops.block_norm_fwd(t["X"], t["Y"], **kw)))
    _, _, r_pre, r_post = ops.block_norm_fwd(t["X"], t["Y"], **kw)
    a = ops.block_norm_bwd(X, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw)
    b = ops.block_norm_bwd(t["X"], t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw)
    assert all(torch.equal(a[i], b[i]) for i in range(4))


def test_norm_in_place_through_the_c_abi(ops):
    from dora_adapter_linear_gb300 import _lib as L
    for M, D in ((45, 1032), (3, 16392)):
        t, kw = norm_case(M, D, BF16, "token", True, seed=8)
        ref = ops.block_norm_fwd(t["X"], t["Y"], **kw)
        sh = L.LoraNormShape(M, D, 1, D, D, D, D, 1.0, 1e-6, 0.0, 1, L.LORA_BF16)
        L.block_norm_fwd(sh, t["X"], t["Y"], kw["w_pre"], kw["w_post"], kw["gate"], t["X"], t["Y"], None, None)
        assert torch.equal(t["X"], ref[0]) and torch.equal(t["Y"], ref[1])


def test_norm_without_rows(ops):
    t, kw = norm_case(0, 64, BF16, "none", True)
    Xout, H, r_pre, r_post = ops.block_norm_fwd(t["X"], t["Y"], **kw)
    assert Xout.shape == H.shape == (0, 64) and r_pre.shape == (0,)
    dX, dY, dw_pre, dw_post, _ = ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw)
    assert dX.shape == dY.shape == (0, 64) and not dw_pre.any() and not dw_post.any()


def test_norm_zero_rows_and_values_that_are_not_finite(ops):
    """A row of zeros has r = eps^-1/2 and finite gradients; inf and NaN stay in their own rows."""
    t, kw = norm_case(20, 256, F32, "token", True, seed=9)
    t["X"][3], t["Y"][3] = 0, 0
    got = ops.block_norm_fwd(t["X"], t["Y"], eps=1e-5, **kw)
    check_norm_fwd(got, t, kw, True, F32, 1e-5)
    check_norm_bwd(ops.block_norm_bwd(got[0], t["Y"], got[2], got[3], t["dH"], t["dXout"], **kw), got[0], t, kw, got[2],
                   got[3], F32)
    t["X"][5, 7], t["Y"][11, 3] = float("nan"), float("inf")
    bad = ops.block_norm_fwd(t["X"], t["Y"], eps=1e-5, **kw)
    rows = [i for i in range(20) if i not in (5, 11)]
    for a, b in zip(bad, got):
        assert torch.equal(a[rows], b[rows])
    assert bad[1][5].isnan().all() and bad[0][11, 3].isnan()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(30, 512), (24, 1024), (1200, 2048), (12, 200)])
def test_norm_rows_that_cancel(ops, M, D, dtype):
    """The block's output nearly takes the residual stream away: the sum of z^2 is far below those of
    its terms, and r_pre keeps the precision of z itself."""
    t, kw = norm_case(M, D, dtype, "none", True, seed=12)
    p = f64(ops.block_norm_fwd(torch.zeros_like(t["X"]), t["Y"], **kw)[0].float())
    keep = torch.from_numpy(np.where(np.arange(M) % 3 == 0, 1.0, np.where(np.arange(M) % 3 == 1, 0.97, 0.0)))
    t["X"] = (-torch.from_numpy(p) * keep[:, None]).to(dtype).to(DEV) + 0.002 * t["X"]
    check_norm_fwd(ops.block_norm_fwd(t["X"], t["Y"], eps=1e-5, **kw), t, kw, True, dtype, 1e-5)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(6, 200), (30, 512), (1200, 2048)])
def test_norm_large_output_with_a_large_weight(ops, M, D, dtype):
    """sum (w_post y)^2 is past the fp32 range, sum y^2 and sum z^2 are not."""
    t, kw = norm_case(M, D, dtype, "none", True, seed=21)
    t["Y"] = t["Y"] * 1e16
    kw["w_post"] = kw["w_post"] * 1e4
    check_norm_fwd(ops.block_norm_fwd(t["X"], t["Y"], eps=1e-5, **kw), t, kw, True, dtype, 1e-5)


@pytest.mark.parametrize("M,D", [(1, 512), (7, 512), (300, 4104), (40, 20488)])
@pytest.mark.parametrize("per", [8192, 1 << 40, 1 << 60, (1 << 63) - 1])
def test_norm_one_gate_row_for_more_rows_than_there_are(ops, M, D, per):
    t, kw = norm_case(M, D, F32, "row", True, seed=22)
    wide = {**kw, "rows_per_gate": per}
    one, other = (ops.block_norm_fwd(t["X"], t["Y"], **k) for k in (kw, wide))
    grads = [ops.block_norm_bwd(one[0], t["Y"], one[2], one[3], t["dH"], t["dXout"], **k) for k in (kw, wide)]
    for a, b in zip((*one, *grads[0]), (*other, *grads[1])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,D", [(13, 8), (77, 64), (501, 40), (50, 72), (333, 128), (9, 256), (8000, 264),
                                 (5001, 384)])
def test_norm_forward_of_short_rows(ops, M, D, dtype):
    """Several rows a warp, of which some take the plain sum and some the one from its terms."""
    test_norm_rows_that_cancel(ops, M, D, dtype)
    test_norm_large_output_with_a_large_weight(ops, M, D, dtype)


def test_norm_gradient_against_differences(ops):
    """fp32: the step's directional derivative by central differences of the forward itself."""
    t, kw = norm_case(24, 128, F32, "seq", True, seed=10, rpg=5, alpha=0.6)
    Xout, H, r_pre, r_post = ops.block_norm_fwd(t["X"], t["Y"], **kw)
    dX, dY, dw_pre, dw_post, dgate = ops.block_norm_bwd(Xout, t["Y"], r_pre, r_post, t["dH"], t["dXout"], **kw)
    gen = torch.Generator(device=DEV).manual_seed(3)
    step = 2.0 ** -7        # the third-order term is about step^2, fp32 rounding about 2^-24 sqrt(M D) / step
    for name, grad in (("X", dX), ("Y", dY), ("w_pre", dw_pre), ("w_post", dw_post), ("gate", dgate)):
        base = t[name] if name in t else kw[name]
        v = torch.randn(base.shape, generator=gen, device=DEV)

        def loss(s):
            a = {**t, name: base + s * v} if name in t else t
            k = kw if name in t else {**kw, name: base + s * v}
            z, h, _, _ = ops.block_norm_fwd(a["X"], a["Y"], **k)
            return float((z.double() * t["dXout"].double()).sum() + (h.double() * t["dH"].double()).sum())

        slope, want = (loss(step) - loss(-step)) / (2 * step), float((grad.double() * v.double()).sum())
        scale = float(grad.double().norm() * v.double().norm())
        assert abs(slope - want) <= 1e-3 * scale, (name, slope, want)


def test_norm_on_another_stream(ops):
    t, kw = norm_case(2048, 1024, BF16, "row", True, seed=11)
    ref = ops.block_norm_fwd(t["X"], t["Y"], **kw)
    rb = ops.block_norm_bwd(ref[0], t["Y"], ref[2], ref[3], t["dH"], t["dXout"], **kw)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = ops.block_norm_fwd(t["X"], t["Y"], **kw)
        gb = ops.block_norm_bwd(got[0], t["Y"], got[2], got[3], t["dH"], t["dXout"], **kw)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got + gb, ref + rb))


# ------------------------------------------------------------------ rotary positions
def turns_of(pos, plan):
    """Exact fractions of a turn [M, rot / 2] of integer positions."""
    bits = [b % 2 ** 64 for b in plan.freq.tolist()]
    return np.array([[(int(p) * b % 2 ** 64) / 2.0 ** 64 for b in bits] for p in pos.tolist()])


def check_rotary(got, x, pos, plan, layout, inverse, dtype):
    t = turns_of(pos, plan)
    ref = BO.rotary(x, t, layout, plan.scale, inverse)
    rot = plan.rot_dim
    size = np.abs(BO.rotary(np.abs(x) + 0j, np.zeros_like(t), layout, abs(plan.scale)).real)
    a = np.abs(x[..., :rot])
    both = (a[..., :rot // 2] + a[..., rot // 2:]) if layout == "half" else (a[..., 0::2] + a[..., 1::2])
    both = np.concatenate((both, both), -1) if layout == "half" else np.repeat(both, 2, -1)
    # angle within pi 2^-25 of the true one (under 2 roundings), sincospi 2 ulp, the factor, two products and a sum
    slack = np.zeros_like(size)
    slack[..., :rot] = 8 * E32 * abs(plan.scale) * both
    within(got[..., :rot], ref[..., :rot], slack[..., :rot], dtype, "rotated")
    assert np.array_equal(to64(got[..., rot:]), x[..., rot:])


ROTARY_CASES = [  # M, H, head_dim, rot_dim, longest position
    (1, 1, 2, 2, 10), (1, 40, 128, 128, 1 << 17), (7, 5, 64, 64, 4096), (33, 3, 80, 32, 1 << 20), (130, 12, 72, 18, 5000),
    (64, 10, 96, 96, 1 << 31), (19, 4, 256, 64, 1 << 40), (5, 2, 20, 12, 100), (300, 8, 128, 64, 1 << 16),
    (3, 1, 514, 514, 77), (50, 64, 64, 16, 999), (257, 2, 128, 120, 2000),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("M,H,hd,rot,longest", ROTARY_CASES)
def test_rotary(ops, M, H, hd, rot, longest, layout, dtype):
    gen = torch.Generator().manual_seed(M * hd + rot)
    x = torch.randn(M, H, hd, generator=gen).to(dtype).to(DEV)
    pos = torch.randint(-3, longest, (M,), generator=gen).to(DEV)
    plan = ops.rotary_plan(rot, 500000.0, layout, "yarn", factor=4.0, device=DEV)
    for call, inverse in ((ops.rotary_fwd, False), (ops.rotary_bwd, True)):
        got = call(x, pos, plan)
        check_rotary(got, f64(x), pos, plan, layout, inverse, dtype)
        # in place in the middle of a packed row: the same bits, and nothing else touched
        row = torch.full((M, (H + 2) * hd), 7.0, dtype=dtype, device=DEV)
        view = row[:, hd:(H + 1) * hd].view(M, H, hd)
        view.copy_(x)
        assert call(view, pos, plan, out=view) is view
        assert torch.equal(view, got) and bool((row[:, :hd] == 7).all()) and bool((row[:, (H + 1) * hd:] == 7).all())
        if longest <= 1 << 31:
            assert torch.equal(call(x, pos.int(), plan), got)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("shift", [1, 2, 4])
def test_rotary_unaligned_and_transposed_heads(ops, layout, shift):
    """Heads at an odd element offset, and a [heads, tokens, head_dim] tensor seen as tokens first."""
    M, H, hd = 21, 3, 64
    plan = ops.rotary_plan(48, layout=layout, device=DEV)
    pos = torch.arange(M, device=DEV) * 1000
    x = torch.randn(M, H, hd, device=DEV).to(BF16)
    ref = ops.rotary_fwd(x, pos, plan)
    flat = torch.zeros(M * 250 + 16, dtype=BF16, device=DEV)
    odd = flat[shift:shift + M * 250].view(M, 250)[:, :H * hd].view(M, H, hd)
    odd.copy_(x)
    assert torch.equal(ops.rotary_fwd(odd, pos, plan), ref)
    assert torch.equal(ops.rotary_fwd(odd, pos, plan, out=odd), ref)
    by_head = x.transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.zeros_like(by_head.transpose(0, 1)).transpose(0, 1)
    assert torch.equal(ops.rotary_fwd(by_head, pos, plan, out=out), ref)
    shared = x[:, :1].expand(M, H, hd)         # one head read H times
    assert torch.equal(ops.rotary_fwd(shared, pos, plan), ref[:, :1].expand(M, H, hd))


def test_rotary_past_32_bit_offsets(ops):
    M, H, hd, ld = 3, 2, 64, (1 << 30) + 8
    big = torch.zeros(2 * ld + H * hd, dtype=BF16, device=DEV)
    plan, pos = ops.rotary_plan(hd, device=DEV), torch.tensor([5, 1 << 33, -9], device=DEV)
    x = torch.randn(M, H, hd, device=DEV).to(BF16)
    view = big.as_strided((M, H, hd), (ld, hd, 1))
    view.copy_(x)
    ref = ops.rotary_fwd(x, pos, plan)
    assert torch.equal(ops.rotary_fwd(view, pos, plan), ref)
    ops.rotary_fwd(view, pos, plan, out=view)
    assert torch.equal(view, ref)


def test_rotary_backward_is_the_transpose_and_no_tokens(ops):
    plan = ops.rotary_plan(64, scaling="yarn", factor=8.0, device=DEV)
    x, g = torch.randn(40, 6, 96, device=DEV), torch.randn(40, 6, 96, device=DEV)
    pos = torch.randint(0, 10000, (40,), device=DEV)
    y, gx = ops.rotary_fwd(x, pos, plan), ops.rotary_bwd(g, pos, plan)
    a, b = float((y.double() * g.double()).sum()), float((x.double() * gx.double()).sum())
    assert abs(a - b) <= 16 * E32 * plan.scale * float((x.double().abs() * g.double().abs()).sum()) * 2
    e = torch.zeros(40, 6, 96, device=DEV)
    e[..., 5] = 1.0             # the map is linear: its difference quotient in a direction is its value there
    step = 0.25
    quotient = (ops.rotary_fwd(x + step * e, pos, plan) - ops.rotary_fwd(x - step * e, pos, plan)) / (2 * step)
    assert float((quotient.double() * g.double()).sum()) == pytest.approx(float(gx[..., 5].double().sum()), abs=1e-3)
    none = torch.empty(0, 6, 96, device=DEV)
    assert ops.rotary_fwd(none, pos[:0], plan).shape == (0, 6, 96)


def test_rotary_refuses_outputs_that_overlap_themselves(ops):
    from dora_adapter_linear_gb300 import LoraError
    plan, pos = ops.rotary_plan(64, device=DEV), torch.arange(4, device=DEV)
    x = torch.randn(4, 2, 64, device=DEV)
    with pytest.raises(LoraError):
        ops.rotary_fwd(x, pos, plan, out=torch.zeros(4, 1, 64, device=DEV).expand(4, 2, 64))
    with pytest.raises(LoraError):
        ops.rotary_fwd(x, pos, plan, out=x.view(2, 4, 64).transpose(0, 1))      # x's memory in another order


# ------------------------------------------------------------------ AdamW
SHAPES = [(16, 520), (8, 1000), (3, 7), (1,), (777,), (256,), (257,), (0,), (40, 64)]


def adamw_set(dtypes, seed, unaligned=False, shapes=SHAPES):
    gen = torch.Generator().manual_seed(seed)
    params, grads = [], []
    for i, s in enumerate(shapes):
        dt = dtypes[i % len(dtypes)]
        n = int(np.prod(s))
        for to, scale in ((params, 0.05), (grads, 0.01)):
            buf = torch.zeros(n + 3, dtype=dt, device=DEV)
            v = buf[1 + i % 3:1 + i % 3 + n] if unaligned else torch.zeros(n, dtype=dt, device=DEV)
            to.append(v.view(s).copy_((torch.randn(n, generator=gen) * scale).to(dt).view(s)))
    return params, grads


def rows(flat, params):
    """The part of a state array that belongs to each tensor."""
    out, row = [], 0
    for p in params:
        out.append(flat.reshape(-1)[row * 256:row * 256 + p.numel()].view(p.shape))
        row += -(-p.numel() // 256)
    return out


@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (BF16, F32)], ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("master", [True, False])
@pytest.mark.parametrize("unaligned", [False, True])
def test_adamw_steps(optim, dtypes, master, unaligned):
    params, _ = adamw_set(dtypes, 1, unaligned)
    muls, decay = [1.0 + i % 3 for i in range(len(params))], [0.1 * (i % 2) for i in range(len(params))]
    opt = optim.AdamW(params, lr=0.01, betas=(0.8, 0.95), eps=1e-6, weight_decay=decay, lr_mul=muls, master=master)
    exact = [f64(p) for p in params]
    m, v = [np.zeros_like(p) for p in exact], [np.zeros_like(p) for p in exact]
    slack = [np.zeros_like(p) for p in exact]
    for t in range(1, 5):
        _, grads = adamw_set(dtypes, 10 + t, unaligned)
        assert opt.step(grads) is None
        for i, g in enumerate(grads):
            lr = 0.01 * muls[i]
            if params[i].dtype == BF16 and not master:      # starts from what the last step stored
                exact[i], slack[i] = stored[i] if t > 1 else exact[i], np.zeros_like(exact[i])
            p0 = exact[i]
            exact[i], m[i], v[i] = BO.adamw(p0, f64(g), m[i], v[i], t, lr, (0.8, 0.95), 1e-6, decay[i])
            # the state within 8 roundings a step of its terms (no cancellation in v; m's terms bounded by
            # their sizes); the update 32 of its own magnitude, in which |m| is at most the sum of its terms
            size = sum(np.abs(x) for x in (p0, exact[i]))
            msum = 0.01 * 6 + np.abs(m[i])
            den = np.sqrt(v[i] / (1 - 0.95 ** t)) + 1e-6
            slack[i] = slack[i] + E32 * (4 * size + 32 * lr * msum / (1 - 0.8 ** t) / den)
        for k, (p, mm, vv) in enumerate(zip(params, rows(opt.m, params), rows(opt.v, params))):
            within(p, exact[k], slack[k] + (UNIT[BF16] * slack[k]), p.dtype, f"p{k} step {t}")
            assert (np.abs(to64(mm) - m[k]) <= 8 * t * E32 * 0.06).all()
            assert (np.abs(to64(vv) - v[k]) <= 8 * t * E32 * v[k] + 1e-45).all()
        if opt.master is not None:
            for k, x in enumerate(rows(opt.master, params)):
                if params[k].dtype == BF16:
                    within(x, exact[k], slack[k], F32, f"master{k}")
                    assert torch.equal(x.to(BF16), params[k])
        stored = [f64(p) for p in params]
        assert opt.steps == t
    used = torch.zeros_like(opt.m)
    for x in rows(used, params):
        x.fill_(1)
    for flat in (opt.m, opt.v):
        assert not flat[used == 0].any()       # what lies past a tensor's end stays zero


@pytest.mark.parametrize("unaligned", [False, True])
@pytest.mark.parametrize("shapes", [SHAPES, [(5,)] * 700], ids=["few", "700"])
def test_adamw_masters_are_the_parameters(optim, unaligned, shapes):
    params, _ = adamw_set((BF16, F32, BF16), 12, unaligned, shapes)
    opt = optim.AdamW(params)
    left = opt.master.clone()
    for p, m, rest in zip(params, rows(opt.master, params), rows(left, params)):
        assert torch.equal(m, p.float()) if p.dtype == BF16 else not m.any()
        rest.zero_()
    assert not left.any()


def encode_like(x, low):
    """The 8-bit blocks of fp32 values [blocks, 256], operation for operation."""
    top = x.abs().amax(1, keepdim=True)
    q = x * torch.where(top > 0, top.reciprocal() * 448.0, torch.zeros(()))
    q = torch.where(x > 0, q.clamp_min(low), q).clamp(-448, 448)
    return q.to(torch.float8_e4m3fn), top * torch.tensor(1.0 / 448.0)


def test_adamw_8bit_states_bit_for_bit(optim):
    """m, v, their codes and scales are a fixed sequence of fp32 operations: equal on the CPU."""
    params, _ = adamw_set((BF16, F32), 2)
    opt = optim.AdamW(params, lr=0.01, weight_decay=0.0, state_bits=8)
    c = lambda x: torch.tensor(x, dtype=torch.float32)  # noqa: E731
    b1, c1, b2, c2 = c(0.9), c(1 - 0.9), c(0.999), c(1 - 0.999)
    cpu = {"m": opt.m.cpu(), "v": opt.v.cpu(), "ms": opt.m_scale.cpu(), "vs": opt.v_scale.cpu()}
    for t in range(1, 5):
        _, grads = adamw_set((BF16, F32), 20 + t)
        if t == 3:
            grads[0].mul_(1e-4)     # a block whose values span many powers of two
            grads[4].zero_()
        opt.step(grads)
        flat = torch.zeros(opt.m.shape)
        for dst, g in zip(rows(flat, params), grads):
            dst.copy_(g.float().cpu())
        m = cpu["m"].float() * cpu["ms"]
        v = cpu["v"].float() * cpu["vs"]
        m = b1 * m + c1 * flat
        v = b2 * (v * v) + (c2 * flat) * flat
        cpu["m"], cpu["ms"] = encode_like(m, -448.0)
        cpu["v"], cpu["vs"] = encode_like(v.sqrt(), 2.0 ** -9)
        for name, got in (("m", opt.m), ("v", opt.v), ("ms", opt.m_scale), ("vs", opt.v_scale)):
            assert torch.equal(got.cpu().float(), cpu[name].float()), (name, t)
        kept = cpu["v"].float()[v > 0]
        assert kept.min() >= 2.0 ** -9       # no second moment above zero is lost


def test_adamw_8bit_first_step_parameters(optim):
    """From a zero state the first step's update is that of exact states."""
    params, grads = adamw_set((F32,), 3)
    before = [f64(p) for p in params]
    optim.AdamW(params, lr=0.01, weight_decay=0.1, state_bits=8).step(grads)
    for k, (p, g, b) in enumerate(zip(params, grads, before)):
        z = np.zeros_like(b)
        ref, _, _ = BO.adamw(b, f64(g), z, z, 1, 0.01, weight_decay=0.1)
        within(p, ref, E32 * (4 * np.abs(b) + 32 * 0.01), F32, f"p{k}")


def test_adamw_8bit_follows_32bit(optim):
    """A quadratic from the same start: both go down, 8-bit states to within a tenth of the way."""
    gen = torch.Generator().manual_seed(5)
    goal = torch.randn(4096, generator=gen).to(DEV)
    loss = {}
    for bits in (32, 8):
        p = torch.zeros(4096, device=DEV)
        opt = optim.AdamW([p], lr=0.02, weight_decay=0.0, state_bits=bits)
        for _ in range(100):
            opt.step([p - goal])
        loss[bits] = float((p - goal).square().mean())
    start = float(goal.square().mean())
    assert loss[32] < 0.2 * start and abs(loss[8] - loss[32]) < 0.1 * start


@pytest.mark.parametrize("shapes", [SHAPES, [(33, 40)] * 700, [(5,)] * 100], ids=["few", "700", "100"])
def test_adamw_clip(optim, shapes):
    """The global norm over one or several launches, the clipped step, and sets beyond one table."""
    params, grads = adamw_set((BF16, F32), 6, shapes=shapes)
    other = [p.clone() for p in params]
    norm = np.sqrt(sum((f64(g) ** 2).sum() for g in grads))
    opt = optim.AdamW(params, lr=0.01)
    got = opt.step(grads, max_norm=0.5 * norm, grad_scale=2.0)      # twice the gradients, a clip to a quarter
    assert abs(float(got) - 2 * norm) <= 64 * E32 * 2 * norm
    ref = optim.AdamW(other, lr=0.01)
    ref.step(grads, grad_scale=0.5)
    for a, b in ((opt.m, ref.m), (opt.v, ref.v)):
        assert float((a.double() - b.double()).abs().max()) <= 256 * E32 * float(b.abs().max()) + 1e-6 / norm * float(b.abs().max())
    assert opt.steps == ref.steps == 1
    assert abs(float(opt.step(grads, max_norm=4 * norm)) - norm) <= 64 * E32 * norm      # below the clip
    assert opt.steps == 2


def test_adamw_skips_gradients_that_are_not_finite_and_none(optim):
    params, grads = adamw_set((BF16, F32), 7)
    opt = optim.AdamW(params, lr=0.01)
    opt.step(grads, max_norm=1.0)
    kept = [t.clone() for t in params + [opt.m, opt.v, opt.master]]
    for bad in (float("inf"), float("nan")):
        worse = [g.clone() for g in grads]
        worse[4][100] = bad
        norm = opt.step(worse, max_norm=float("inf"))
        assert not bool(norm.isfinite()) and opt.steps == 1
        assert all(torch.equal(a, b) for a, b in zip(params + [opt.m, opt.v, opt.master], kept))
    part = [g if i % 2 else None for i, g in enumerate(grads)]
    norm = opt.step(part, max_norm=1e9)
    assert opt.steps == 2
    want = np.sqrt(sum((f64(g) ** 2).sum() for g in part if g is not None))
    assert abs(float(norm) - want) <= 64 * E32 * want
    for i, (p, k) in enumerate(zip(params, kept)):
        assert p.numel() == 0 or torch.equal(p, k) == (i % 2 == 0)
    assert float(opt.step([None] * len(params), max_norm=1.0)) == 0.0 and opt.steps == 2


def test_adamw_in_a_graph_counts_its_replays(optim):
    params, grads = adamw_set((BF16,), 8)
    twin = [p.clone() for p in params]
    a, b = optim.AdamW(params, lr=1.0), optim.AdamW(twin, lr=1.0)
    rate = torch.tensor(0.01, device=DEV)
    a.step(grads, lr=rate, max_norm=1.0)        # also makes the workspace
    b.step(grads, lr=0.01, max_norm=1.0)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        a.step(grads, lr=rate, max_norm=1.0)
    side.synchronize()
    b.step(grads, lr=0.01, max_norm=1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.step(grads, lr=rate, max_norm=1.0)
    for lr in (0.01, 0.005, 0.0025):
        rate.fill_(lr)
        graph.replay()
        b.step(grads, lr=lr, max_norm=1.0)
    torch.cuda.synchronize()
    assert a.steps == b.steps == 5
    assert all(torch.equal(x, y) for x, y in zip(params + [a.m, a.v, a.master], twin + [b.m, b.v, b.master]))


def test_adamw_state_dict_and_refusals(optim):
    params, grads = adamw_set((BF16, F32), 9)
    for bits in (32, 8):
        a = optim.AdamW([p.clone() for p in params], state_bits=bits)
        a.step(grads)
        b = optim.AdamW([p.clone() for p in a.params], state_bits=bits)
        b.load_state_dict({k: v.clone() if hasattr(v, "clone") else v for k, v in a.state_dict().items()})
        a.step(grads)
        b.step(grads)
        assert a.steps == b.steps == 2 and all(torch.equal(x, y) for x, y in zip(a.params, b.params))
        with pytest.raises(ValueError):
            optim.AdamW([p.clone() for p in params], state_bits=40 - bits).load_state_dict(a.state_dict())
        with pytest.raises(ValueError):
            optim.AdamW(params[:2], state_bits=bits).load_state_dict(a.state_dict())
    swapped = optim.AdamW([torch.zeros(512, device=DEV), torch.zeros(100, device=DEV)])
    with pytest.raises(ValueError):     # as many blocks, other tensors
        swapped.load_state_dict(optim.AdamW([torch.zeros(100, device=DEV), torch.zeros(512, device=DEV)]).state_dict())
    flat = torch.zeros(100, device=DEV)
    for shared in ([flat, flat], [flat[:60], flat[50:]]):
        with pytest.raises(ValueError):
            optim.AdamW(shared)
    optim.AdamW([flat[:50], flat[50:], flat[:0]])
    opt = optim.AdamW(params)
    wrong = [grads[:-1], [grads[0].float()] + grads[1:], [grads[0].t().contiguous()] + grads[1:],
             [grads[0].cpu()] + grads[1:], [torch.zeros(520, 16, dtype=BF16, device=DEV).t()] + grads[1:]]
    for g in wrong:
        with pytest.raises(ValueError):
            opt.step(g)
    for kw in (dict(max_norm=0.0), dict(max_norm=float("nan")), dict(lr=torch.zeros(2, device=DEV)),
               dict(lr=torch.zeros(())), dict(lr=torch.zeros((), dtype=torch.float64, device=DEV))):
        with pytest.raises(ValueError):
            opt.step(grads, **kw)
    assert opt.steps == 0
    for kw in (dict(state_bits=16), dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=0.0), dict(lr_mul=[1.0]),
               dict(weight_decay=float("nan")), dict(params=[params[0].t()])):
        with pytest.raises(ValueError):
            optim.AdamW(**{"params": params, **kw})
