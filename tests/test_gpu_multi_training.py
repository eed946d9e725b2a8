"""Several adapters trained in one batch and then decoded with: plan, forward, backward, clipping by adapter and
AdamW together, every stage against its reference on the numbers that it got."""
import numpy as np
import pytest
import torch

import multi_cases as C
from dora_adapter_linear_gb300 import ops, optim
from oracle import block_oracle, multi_oracle as O

pytestmark = pytest.mark.gpu


def step(g, dY, opt, max_norm):
    """One training step of all adapters; what it left behind, by name."""
    n = g["A"].shape[0]
    plan = ops.adapter_plan(g["ids"], n)
    Y, Z = ops.lora_multi_fwd(g["X"], g["W0"], g["A"], g["B"], g["s"], plan, bias=g["bias"])
    dX, dA, dB, db = ops.lora_multi_bwd(g["X"], g["W0"], g["A"], g["B"], Z, dY, g["s"], plan, need_dbias=True)
    out = {"Y": Y, "Z": Z, "dX": dX, "dA": dA.clone(), "dB": dB.clone(), "dbias": db}
    out["norms"] = optim.clip_grads([dA, dB], max_norm, groups=n)
    out["cA"], out["cB"] = dA, dB
    opt.step([dA, dB])
    return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_training_steps_and_decoding(dtype):
    M, d_in, d_out, r, n = 330, 136, 264, 16, 5
    c = C.inputs(M, d_in, d_out, r, n, "runs", dtype)
    c["ids"] = np.repeat([0, 2, 4, -1, 2, 1], 55)        # adapter 3 has no rows
    g = {k: v.cuda() if torch.is_tensor(v) else torch.from_numpy(v).cuda() for k, v in c.items()}
    opt = optim.AdamW([g["A"], g["B"]], lr=0.01, weight_decay=[0.01, 0.0], master=False)
    m = [np.zeros(t.numel()) for t in (g["A"], g["B"])]
    v = [np.zeros(t.numel()) for t in (g["A"], g["B"])]
    sizes = [np.zeros(t.numel()) for t in (g["A"], g["B"])]       # m with the terms' magnitudes
    for k in range(3):
        c.update(A=g["A"].cpu().clone(), B=g["B"].cpu().clone())
        dY = torch.randn(M, d_out, generator=torch.Generator().manual_seed(k)).mul_(0.1).to(g["X"].dtype)
        c["dY"] = dY
        out = step(g, dY.cuda(), opt, 1.5)
        ref = {**C.reference_fwd(c, dtype), **C.reference_bwd(c, out["Z"], dtype)}
        for name, value in ref.items():
            C.near(out[name], value, f"{name} of step {k}")
        assert not out["dA"][3].any() and not out["dB"][3].any()
        entries = [C.f64(out[name][a]) for name in ("dA", "dB") for a in range(n)]
        norms, clipped = O.clip(entries, 1.5, list(range(n)) * 2, n)
        assert (abs(C.f64(out["norms"]) - norms) <= 48 * 2.0 ** -24 * norms).all()
        half = C.half_step(dtype) + 56 * 2.0 ** -24
        for i, want in enumerate(clipped):
            got = C.f64(out["cA" if i < n else "cB"][i % n])
            assert (abs(got - want) <= half * abs(want) + 1e-30).all()
        for i, (p, grad) in enumerate((("A", "cA"), ("B", "cB"))):
            old, grad = C.f64(c[p]).ravel(), C.f64(out[grad]).ravel()
            want, m[i], v[i] = block_oracle.adamw(old, grad, m[i], v[i], k + 1, 0.01, weight_decay=[0.01, 0.0][i])
            sizes[i] = 0.9 * sizes[i] + 0.1 * abs(grad)
            # 32 roundings of 2^-24 of the update's terms (the state takes up to 8 a step), 4 of the parameter's, and
            # its own rounding where it is stored
            den = np.sqrt(v[i] / (1 - 0.999 ** (k + 1))) + 1e-8
            off = 2.0 ** -24 * (4 * (abs(old) + abs(want)) + 32 * 0.01 * sizes[i] / (1 - 0.9 ** (k + 1)) / den)
            off += C.half_step(dtype) * (abs(want) + off)
            assert (abs(C.f64(g[p]).ravel() - want) <= off).all(), p
    # decoded one row, and a few rows, at a time: the trained adapters' outputs
    c.update(A=g["A"].cpu(), B=g["B"].cpu())
    want = C.reference_fwd(c, dtype)["Y"]
    for rows in ([0], [60], [329], list(range(40, 75)), list(range(0, 330, 7))):
        at = torch.tensor(rows, device="cuda")
        plan = ops.adapter_plan(g["ids"][at], n)
        Y, _ = ops.lora_multi_fwd(g["X"][at].contiguous(), g["W0"], g["A"], g["B"], g["s"], plan, bias=g["bias"], save_z=False)
        C.near(Y, (want[0][rows], want[1][rows]), f"rows {rows[0]} and on")


def test_one_adapter_that_diverges_leaves_the_others_alone():
    c = C.inputs(300, 136, 264, 16, 4, "rows", "bf16")
    runs = []
    for sick in (False, True):
        g = {k: v.cuda() if torch.is_tensor(v) else torch.from_numpy(np.asarray(v)).cuda() for k, v in c.items()}
        opt = optim.AdamW([g["A"], g["B"]], lr=0.01, weight_decay=0.0, master=False)
        dY = g["dY"].clone()
        if sick:
            dY[g["ids"] == 1] = float("inf")
        runs.append((g, step(g, dY, opt, 1.0)))
    (g0, _), (g1, out) = runs
    assert out["norms"].isfinite().tolist() == [True, False, True, True]
    for name in ("A", "B"):
        for a in (0, 2, 3):
            assert torch.equal(g0[name][a], g1[name][a])
        assert torch.equal(g1[name][1].cpu(), c[name][1])           # no step, no decay
