"""Inputs, reference and tolerances of the many-adapter tests (not a test module).

An output's error is at most: half a step of its type; for every sum of k products formed in fp32, k + 4 steps
of 2^-23 of the sum of the products' magnitudes (a tensor core's sums may be cut off instead of rounded, so a
whole step each); and, with bf16, half a step (2^-8) of the rank-r values (s z, or s g) that enter the second
product rounded.  As a factor of dA, s g comes in two parts, the second what the first one's rounding left: half
a step of half a step."""
import numpy as np
import torch

from oracle import multi_oracle as O

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = 2.0 ** -23


def ids_of(style, M, n, rng):
    if style == "one":
        return np.zeros(M, np.int64) + n - 1
    if style == "none":
        return np.full(M, -1)
    if style == "rows":
        return rng.integers(0, n, M)
    if style == "bare":                                  # some rows, and some ids outside of the range
        return rng.choice(np.concatenate((np.arange(n), [-1, n, -7])), M)
    assert style == "runs"
    cuts = np.sort(rng.integers(0, M + 1, min(9, M)))
    return np.concatenate([np.full(len(p), rng.integers(-1, n)) for p in np.split(np.arange(M), cuts)])


def inputs(M, d_in, d_out, r, n, style, dtype, seed=0, bias=True):
    """CPU tensors of one case by name; `ids` as numbers."""
    gen, rng = torch.Generator().manual_seed(seed), np.random.default_rng(seed)
    normal = lambda *s: torch.randn(*s, generator=gen).to(DTYPES[dtype])  # noqa: E731
    return {"X": normal(M, d_in), "W0": normal(d_out, d_in), "A": normal(n, r, d_in), "B": normal(n, d_out, r),
            "s": torch.rand(n, generator=gen) * 2 - 0.5, "bias": normal(d_out) if bias else None,
            "dY": normal(M, d_out), "ids": ids_of(style, M, n, rng) if M else np.zeros(0, np.int64)}


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(DTYPES[dtype]).eps / 2


def reference_fwd(c, dtype):
    """{name: (value, most that it may be off)}"""
    X, W0, A, B, s = (f64(c[k]) for k in ("X", "W0", "A", "B", "s"))
    d_in, r, h, bias = X.shape[1], A.shape[1], half_step(dtype), f64(c["bias"])
    Y, Z = O.multi_fwd(X, W0, A, B, s, c["ids"], bias)
    mY, mZ = O.multi_fwd(abs(X), abs(W0), abs(A), abs(B), abs(s), c["ids"], None if bias is None else abs(bias))
    zero = np.zeros_like(W0)
    lora = O.multi_fwd(X, zero, A, B, s, c["ids"])[0] * 0
    for i, a in enumerate(c["ids"]):                     # the update with its z rounded
        if 0 <= a < len(A):
            lora[i] = abs(s[a]) * (abs(B[a]) @ abs(Z[i]))
    off_z = (d_in + 4) * STEP * mZ
    off = (d_in + r + 8) * STEP * mY + (half_step("bf16") * lora if dtype == "bf16" else 0)
    return {"Y": (Y, h * (abs(Y) + off) + off), "Z": (Z, h * (abs(Z) + off_z) + off_z)}


def reference_bwd(c, Z, dtype):
    X, W0, A, B, s, dY, Z = (f64(c[k]) if isinstance(k, str) else k for k in ("X", "W0", "A", "B", "s", "dY", f64(Z)))
    M, (d_out, r), h = X.shape[0], B.shape[1:], half_step(dtype)
    dX, dA, dB, db, G = O.multi_bwd(X, W0, A, B, s, c["ids"], Z, dY)
    mX, mA, mB, mb, _ = O.multi_bwd(abs(X), abs(W0), abs(A), abs(B), abs(s), c["ids"], abs(Z), abs(dY))
    round_g = half_step("bf16") if dtype == "bf16" else 0
    rX, rA, _, _, _ = O.multi_bwd(abs(X), 0 * W0, abs(A), 0 * B, abs(s), c["ids"], abs(Z), 0 * dY)
    for i, a in enumerate(c["ids"]):                     # the terms with their g rounded
        if 0 <= a < len(A):
            rX[i] = abs(G[i]) @ abs(A[a])
            rA[a] += np.outer(abs(G[i]), abs(X[i]))
    offs = {"dX": (d_out + r + 8) * STEP * mX + round_g * rX, "dA": (2 * M + d_out + 8) * STEP * mA + round_g ** 2 * rA,
            "dB": (M + 8) * STEP * mB, "dbias": (M + 4) * STEP * mb}
    return {k: (v, h * (abs(v) + offs[k]) + offs[k]) for k, v in (("dX", dX), ("dA", dA), ("dB", dB), ("dbias", db))}


def near(got, ref, what):
    value, off = ref
    got = f64(got)
    assert got.shape == value.shape, what
    wrong = ~(abs(got - value) <= off)
    if wrong.any():
        at = np.unravel_index(np.argmax(np.where(np.isfinite(got), abs(got - value) / np.maximum(off, 1e-300), np.inf)), got.shape)
        raise AssertionError(f"{what}: {wrong.sum()} of {wrong.size} off, worst at {at}: {got[at]} for {value[at]} +- {off[at]}")
