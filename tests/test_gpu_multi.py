"""The many-adapter projection against its fp64 reference, element by element."""
import threading

import numpy as np
import pytest
import torch

from dora_adapter_linear_gb300 import _lib as L
from dora_adapter_linear_gb300 import ops, optim
import multi_cases as C
from oracle import multi_oracle as O

pytestmark = pytest.mark.gpu


def cuda(c):
    g = {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}
    g["ids"] = torch.from_numpy(np.asarray(c["ids"], np.int64)).cuda()
    return g


def fwd(g, plan=None, **kw):
    plan = plan or ops.adapter_plan(g["ids"], g["A"].shape[0])
    return ops.lora_multi_fwd(g["X"], g["W0"], g["A"], g["B"], g["s"], plan, bias=g["bias"], **kw)


def bwd(g, Z, plan=None, **kw):
    plan = plan or ops.adapter_plan(g["ids"], g["A"].shape[0])
    return ops.lora_multi_bwd(g["X"], g["W0"], g["A"], g["B"], Z, g["dY"], g["s"], plan, need_dbias=True, **kw)


SIZES = [  # M, d_in, d_out, r, n, ids
    (0, 64, 72, 8, 3, "one"), (1, 8, 8, 8, 1, "one"), (1, 4096, 72, 16, 4, "rows"), (1, 64, 4104, 16, 2, "none"),
    (2, 264, 1000, 24, 300, "rows"), (7, 72, 8, 128, 5, "bare"), (16, 1000, 264, 16, 16, "rows"), (17, 520, 136, 64, 9, "rows"),
    (31, 512, 512, 40, 3, "runs"), (33, 128, 256, 8, 40, "rows"), (64, 1024, 520, 16, 64, "rows"), (65, 72, 64, 72, 2, "bare"),
    (128, 264, 392, 16, 7, "runs"), (130, 64, 1032, 32, 130, "rows"), (255, 40, 264, 16, 1, "one"), (256, 64, 256, 128, 3, "bare"),
    (257, 520, 8, 8, 600, "rows"), (300, 128, 264, 16, 5, "runs"), (511, 72, 328, 104, 6, "runs"), (513, 200, 72, 56, 4, "runs"),
    (700, 64, 512, 16, 2, "none"), (1029, 72, 136, 24, 3, "runs"), (1500, 16, 24, 64, 100, "rows"), (2600, 24, 40, 8, 2, "one"),
]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,d_in,d_out,r,n,style", SIZES)
def test_forward_and_backward(M, d_in, d_out, r, n, style, dtype):
    r -= 3 if dtype == "f32" and r > 8 else 0            # fp32: any rank
    c = C.inputs(M, d_in, d_out, r, n, style, dtype, seed=M + r)
    g = cuda(c)
    Y, Z = fwd(g)
    ref = C.reference_fwd(c, dtype)
    C.near(Y, ref["Y"], "Y")
    C.near(Z, ref["Z"], "Z")
    grads = dict(zip(("dX", "dA", "dB", "dbias"), bwd(g, Z)))
    for k, v in C.reference_bwd(c, Z, dtype).items():
        C.near(grads[k], v, k)
    ops.check_device_errors()


@pytest.mark.parametrize("M,d_in,d_out,r,n,style", [
    (2570, 1800, 1816, 8, 5, "bare"), (2570, 1816, 1800, 16, 300, "rows"), (2600, 1800, 2048, 24, 9, "runs"),
    (2561, 2568, 1800, 32, 40, "rows"), (2820, 1800, 1832, 32, 1, "one"), (2600, 1800, 1800, 72, 3, "runs")])
def test_products_that_fill_the_device(M, d_in, d_out, r, n, style):
    """Enough tiles for every multiprocessor: the gradients' sums run beside the product.  Z recomputed has the same bits."""
    c = C.inputs(M, d_in, d_out, r, n, style, "bf16", seed=M + r)
    g = cuda(c)
    Y, Z = fwd(g)
    ref = C.reference_fwd(c, "bf16")
    C.near(Y, ref["Y"], "Y")
    C.near(Z, ref["Z"], "Z")
    first = bwd(g, Z)
    grads = dict(zip(("dX", "dA", "dB", "dbias"), first))
    for k, v in C.reference_bwd(c, Z, "bf16").items():
        C.near(grads[k], v, k)
    for other in (Z, None):
        assert all(torch.equal(a, b) for a, b in zip(first, bwd(g, other)))
    ops.check_device_errors()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_options(dtype):
    """No bias, a number as scale, 32-bit ids, no saved Z, no dX, Z recomputed."""
    c = C.inputs(90, 136, 72, 16, 4, "runs", dtype, bias=False)
    g = cuda(c)
    plan = ops.adapter_plan(g["ids"].int(), 4)
    c["s"] = torch.full((4,), 0.75)
    args = g["X"], g["W0"], g["A"], g["B"]
    Y, Z = ops.lora_multi_fwd(*args, 0.75, plan)
    C.near(Y, C.reference_fwd(c, dtype)["Y"], "Y")
    Y2, none = ops.lora_multi_fwd(*args, 0.75, plan, save_z=False)
    assert none is None and torch.equal(Y, Y2)
    dX, dA, dB, db = ops.lora_multi_bwd(*args, Z, g["dY"], 0.75, plan)
    assert db is None
    none, dA2, dB2, db2 = ops.lora_multi_bwd(*args, None, g["dY"], 0.75, plan, need_dx=False, need_dbias=True)
    assert none is None and torch.equal(dA, dA2) and torch.equal(dB, dB2)      # the recomputed Z has the same bits
    ref = C.reference_bwd(c, Z, dtype)
    for k, v in (("dX", dX), ("dA", dA), ("dB", dB), ("dbias", db2)):
        C.near(v, ref[k], k)


@pytest.mark.parametrize("M,r", [(40, 16), (300, 16), (600, 72)])
def test_what_is_not_finite_stays_with_its_adapter(M, r):
    """Adapter 1 holds NaN and infinities, row 5 too: other rows and other adapters' gradients keep their bits."""
    c = C.inputs(M, 136, 264, r, 4, "rows", "bf16")
    g = cuda(c)
    plan = ops.adapter_plan(g["ids"], 4)
    Y0, Z0 = fwd(g, plan)
    d0 = bwd(g, Z0, plan)
    g2 = {k: v.clone() if torch.is_tensor(v) else v for k, v in g.items()}
    g2["A"][1, :, ::3], g2["B"][1, ::2], g2["s"][1] = float("nan"), float("inf"), float("nan")
    bad = c["ids"] == 1
    sick = int(np.flatnonzero(c["ids"] == 2)[1])         # one row of adapter 2
    g2["X"][sick], g2["dY"][sick] = float("inf"), float("nan")
    Y, Z = fwd(g2, plan)
    fine = torch.from_numpy(~bad).cuda()
    fine[sick] = False
    assert torch.equal(Y[fine], Y0[fine]) and torch.equal(Z[fine], Z0[fine])
    assert Y[torch.from_numpy(bad).cuda()].isnan().any(1).all()
    Zb = torch.where(fine[:, None], Z0, float("nan"))
    dX, dA, dB, _ = bwd(g2, Zb, plan)
    assert torch.equal(dX[fine], d0[0][fine])
    for a in (0, 3):
        assert torch.equal(dA[a], d0[1][a]) and torch.equal(dB[a], d0[2][a])


def test_same_bits_again_and_rows_of_any_order():
    """Sums have one order: a call repeats its bits, and a row's output does not depend on its neighbours."""
    c = C.inputs(700, 136, 264, 16, 5, "rows", "bf16")
    g = cuda(c)
    Y, Z = fwd(g)
    first = bwd(g, Z)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, bwd(g, Z)))
    perm = torch.randperm(700, generator=torch.Generator().manual_seed(1)).cuda()
    h = dict(g, X=g["X"][perm], ids=g["ids"][perm])
    Y2, Z2 = fwd(h)
    assert torch.equal(Y2, Y[perm]) and torch.equal(Z2, Z[perm])


@pytest.mark.parametrize("M", [5, 70, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_outside_of_the_outputs_is_written(M, dtype):
    d_in, d_out, r, n = 72, 136, 24, 3
    c = C.inputs(M, d_in, d_out, r, n, "runs", dtype)
    g, dt = cuda(c), C.DTYPES[dtype]
    plan = ops.adapter_plan(g["ids"], n)
    sh = L.LoraMultiShape(M, d_in, d_out, r, n, L.dtype_code(g["X"]))
    sizes = {"Y": M * d_out, "Z": M * r, "dX": M * d_in, "dA": n * r * d_in, "dB": n * d_out * r, "db": d_out}
    bufs = {k: torch.full((v + 512,), 7.0, dtype=dt, device="cuda") for k, v in sizes.items()}
    out = {k: bufs[k][256:256 + v] for k, v in sizes.items()}
    for back in (False, True):
        need = L.lora_multi_workspace_bytes(back, sh)
        ws = torch.full((need + 4096,), 0x55, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        if back:
            L.lora_multi_bwd(sh, g["X"], g["W0"], g["A"], g["B"], out["Z"], g["dY"], g["s"], plan.buffer, out["dX"],
                             out["dA"], out["dB"], out["db"], ws[:need])
        else:
            L.lora_multi_fwd(sh, g["X"], g["W0"], g["A"], g["B"], g["bias"], g["s"], plan.buffer, out["Y"], out["Z"],
                             ws[:need])
        assert (ws[need:] == 0x55).all()
    for k, b in bufs.items():
        assert (b[:256] == 7).all() and (b[256 + sizes[k]:] == 7).all(), k
    Y, Z = fwd(g, plan)
    assert torch.equal(out["Y"].view(M, d_out), Y) and torch.equal(out["Z"].view(M, r), Z)


@pytest.mark.parametrize("rows,n", [(1, 1), (31, 2), (300, 5), (1000, 255), (1000, 256), (5000, 700), (70000, 65535)])
def test_plan(rows, n):
    """Rows by adapter in their own order, items, pieces and tiles."""
    rng = np.random.default_rng(rows)
    ids = rng.integers(-2, n + 2, rows)
    ids[rng.random(rows) < 0.3] = n - 1
    buf = ops.adapter_plan(torch.from_numpy(ids).cuda(), n).buffer.cpu().numpy()
    at = 0

    def take(count, words=1):
        nonlocal at
        v = buf[at:at + 4 * count * words].view(np.int32)
        at += (4 * count * words + 255) // 256 * 256
        return v.reshape(count, words) if words > 1 else v

    used, tiles = min(rows, n), (rows + 255) // 256
    head, kept, order, _, start, istart, pstart = (take(k) for k in (64, rows, rows, rows, n + 1, n + 1, n + 1))
    items, pieces = take(rows // 64 + used, 4), take(rows // 512 + used, 4)
    tcount, tlist, tmask = take(tiles), take(tiles * 256).reshape(tiles, 256), take(tiles * 256 * 8).reshape(tiles, 256, 8)
    assert at == L.lora_multi_plan_bytes(rows, n)
    real = np.where((ids >= 0) & (ids < n), ids, -1)
    assert (kept == real).all()
    key = np.where(real < 0, n, real)
    assert (order == np.argsort(key, kind="stable")).all()
    assert (start == np.searchsorted(np.sort(key), np.arange(n + 1))).all()
    slots = 0
    for first, list_, size in ((istart, items, 64), (pstart, pieces, 512)):
        count = -(-np.diff(start) // size)
        assert (first == np.concatenate(([0], np.cumsum(count)))).all()
        k = 0
        for a in np.flatnonzero(count):
            for b in range(start[a], start[a + 1], size):
                want = [a, b, min(size, start[a + 1] - b), 0]
                if size == 512:
                    want[3] = -1 if count[a] == 1 else slots
                    slots += count[a] > 1
                assert list_[k].tolist() == want
                k += 1
        assert head[0 if size == 64 else 1] == k <= len(list_)
    assert slots <= 2 * (rows // 512) and head[2] == start[n]
    for t in range(tiles):
        mine = np.full(256, -1)
        mine[:len(real[256 * t:256 * t + 256])] = real[256 * t:256 * t + 256]
        seen = list(dict.fromkeys(mine[mine >= 0].tolist()))
        assert tlist[t, :tcount[t]].tolist() == seen
        for k, a in enumerate(seen):
            bits = np.unpackbits(tmask[t, k].copy().view(np.uint8), bitorder="little")
            assert (bits == (mine != a)).all()


def test_captured_step_follows_its_ids():
    """Plan, forward and backward in one graph, replayed with other ids and inputs in the same buffers."""
    for M in (24, 300):
        cases = [C.inputs(M, 72, 136, 16, 4, style, "bf16", seed=k) for k, style in enumerate(("runs", "rows", "none"))]
        g = cuda(cases[0])
        plan = ops.adapter_plan(g["ids"], 4)
        Y, Z = fwd(g, plan)
        bwd(g, Z, plan)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.update(g["ids"])
            Y, Z = fwd(g, plan)
            grads = bwd(g, Z, plan)
        for c in cases[1:] + cases[:1]:
            for k, v in cuda(c).items():
                if torch.is_tensor(v):
                    g[k].copy_(v)
            other = fwd(g)[0]                            # a call beside the graph's
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(other, Y)
            C.near(Y, C.reference_fwd(c, "bf16")["Y"], "Y")
            for k, v in C.reference_bwd(c, Z, "bf16").items():
                C.near(dict(zip(("dX", "dA", "dB", "dbias"), grads))[k], v, k)


def test_a_plan_without_ids_is_refused():
    c = C.inputs(8, 64, 72, 8, 3, "rows", "bf16")
    g = cuda(c)
    plan = ops.AdapterPlan(8, 3, g["X"].device)
    for call in (lambda: fwd(g, plan), lambda: bwd(g, None, plan)):
        with pytest.raises(ValueError, match="no ids yet"):
            call()
    plan.update(g["ids"])
    C.near(fwd(g, plan)[0], C.reference_fwd(c, "bf16")["Y"], "Y")


def test_another_stream():
    c = C.inputs(300, 136, 264, 16, 5, "runs", "bf16")
    g = cuda(c)
    Y0, Z0 = fwd(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y, Z = fwd(g)
        grads = bwd(g, Z)
    side.synchronize()
    assert torch.equal(Y, Y0) and all(torch.equal(a, b) for a, b in zip(grads, bwd(g, Z0)))


def test_offsets_past_32_bits():
    """Stacks of more than 2^31 elements, and as many outputs: the last adapters and rows are right."""
    n, r, d = 1030, 128, 16392
    A, B = torch.zeros(n, r, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 72, r, dtype=torch.bfloat16, device="cuda")
    c = C.inputs(40, d, 72, r, 3, "rows", "bf16")
    A[-3:], B[-3:] = c["A"].cuda(), c["B"].cuda()
    g = dict(cuda(c), A=A, B=B, s=torch.cat((torch.zeros(n - 3), c["s"])).cuda())
    g["ids"] += n - 3
    Y, Z = fwd(g)
    ref = C.reference_fwd(c, "bf16")
    C.near(Y, ref["Y"], "Y")
    C.near(Z, ref["Z"], "Z")
    dX, dA, dB, _ = bwd(g, Z)
    ref = C.reference_bwd(c, Z, "bf16")
    C.near(dX, ref["dX"], "dX")
    C.near(dA[-3:], ref["dA"], "dA")
    C.near(dB[-3:], ref["dB"], "dB")
    assert not dA[:-3].any() and not dB[:-3].any()
    del A, B, g, dA, dB
    M, d_out = 2 ** 18 + 37, 8200
    c = C.inputs(64, 8, d_out, 8, 3, "rows", "bf16")
    g = cuda(c)
    g["X"] = torch.cat((torch.zeros(M - 64, 8, dtype=torch.bfloat16, device="cuda"), g["X"]))
    g["ids"] = torch.cat((torch.full((M - 64,), -1, device="cuda"), g["ids"]))
    Y, Z = fwd(g)
    ref = C.reference_fwd(c, "bf16")
    C.near(Y[-64:], ref["Y"], "Y")
    assert torch.equal(Y[:M - 64:4099], g["bias"].expand(len(Y[:M - 64:4099]), -1))


@pytest.mark.parametrize("M", [3, 40, 300])
def test_infinite_values_stay_infinite(M):
    """A z that overflows gives its row infinities of the formula's signs, as one product would, and no NaN."""
    c = C.inputs(M, 64, 72, 8, 2, "one", "bf16", bias=False)
    c["A"][:], c["B"][:] = 0, 1
    c["A"][1, 3, 5], c["X"][:, 5], c["s"][:] = 2.0 ** 100, 1, 1
    c["X"][1, 5], c["X"][2, 5] = 3e38, -3e38
    g = cuda(c)
    Y, Z = fwd(g)
    # the base's own product of 3e38 overflows too where its weight is above 1.13: the other way, the sum is NaN
    base = g["X"][:3, 5].float()[:, None] * g["W0"][:, 5].float()
    want = base + torch.tensor([0, float("inf"), -float("inf")], device="cuda")[:, None]
    assert Y[0].isfinite().all()
    for i in (1, 2):
        assert torch.equal(Y[i].isnan(), want[i].isnan())
        assert torch.equal(Y[i].float()[~want[i].isnan()], want[i][~want[i].isnan()])
    assert Z[1, 3] == float("inf") and Z[2, 3] == -float("inf")
    g["dY"][:] = 0
    g["dY"][1, 0], g["B"][1, 0] = 1, 0                   # g_1 has one element, which overflows times the scale
    g["B"][1, 0, 2], g["s"][1], g["X"][1] = 3e38, 4.0, 1
    dX, dA, dB, _ = bwd(g, torch.ones_like(Z))
    assert (dA[1, 2] == float("inf")).all() and dA[1, [0, 1, 3]].isfinite().all()


@pytest.mark.parametrize("own_streams", [False, True])
def test_threads(own_streams):
    """Calls of four threads, on one stream, where their launches come in any order, or on one each."""
    cases = [cuda(C.inputs(M, d, d + 16, r, 5, "rows", "bf16", seed=M)) for M, d, r in
             ((5, 520, 16), (150, 136, 24), (700, 264, 8), (2570, 1800, 32))]
    plans = [ops.adapter_plan(g["ids"], 5) for g in cases]

    def step(i):
        Y, Z = fwd(cases[i], plans[i])
        grads = bwd(cases[i], Z, plans[i])
        norms = optim.clip_grads([grads[1], grads[2]], 1.0, groups=5)
        return (Y, Z, norms) + grads

    want = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    wrong = []

    def run(i):
        stream = torch.cuda.Stream() if own_streams else torch.cuda.default_stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                got = step(i)
                stream.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(i)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    ops.check_device_errors()


def same_kinds(got, want, what):
    """NaN and signed infinities where the formula has them."""
    got = C.f64(got)
    for kind in (np.isnan, np.isposinf, np.isneginf):
        assert (kind(got) == kind(want)).all(), f"{what}: {kind.__name__}"


def one_infinity(M, dtype, where):
    """A case of 16 columns of rank and three adapters in turn, and the same with an infinity at each of `where`:
    (name, index, sign).  Values of z and g that meet one are far enough from zero to have a sign."""
    c = C.inputs(M, 72, 136, 16, 3, "rows", dtype, seed=6)
    c["ids"] = np.arange(M) % 3
    X, W0, A, B, s, dY = (C.f64(c[k]) for k in ("X", "W0", "A", "B", "s", "dY"))
    Z = O.multi_fwd(X, W0, A, B, s, c["ids"])[1]
    G = O.multi_bwd(X, W0, A, B, s, c["ids"], Z, dY)[4]
    mZ = O.multi_fwd(abs(X), W0, abs(A), B, s, c["ids"])[1]
    mG = O.multi_bwd(X, W0, A, abs(B), abs(s), c["ids"], Z, abs(dY))[4]
    for at in ((1, slice(None)), (slice(1, None, 3), [3, 9, 15])):
        assert (abs(Z) > 80 * C.STEP * mZ)[at].all() and (abs(G) > 144 * C.STEP * mG)[at].all()
    d = {k: v.clone() if torch.is_tensor(v) else v for k, v in c.items()}
    for name, at, sign in where:
        d[name][at] = sign * float("inf")
    return c, d


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("where", [[("B", (1, 5, 3), 1)], [("B", (1, 5, 3), -1), ("B", (1, 70, 9), 1)], [("B", (1, 135, 15), -1)]])
def test_an_infinity_in_B(M, dtype, where):
    """Its column of the adapter's rows is the infinity of the formula's sign, all else keeps its bits."""
    c, d = one_infinity(M, dtype, where)
    Y0, Z0 = fwd(cuda(c))
    Y, Z = fwd(cuda(d))
    assert torch.equal(Z, Z0)
    with np.errstate(all="ignore"):
        want = O.multi_fwd(*(C.f64(d[k]) for k in ("X", "W0", "A", "B", "s")), c["ids"], C.f64(c["bias"]))[0]
    assert np.isinf(want).sum() == len(where) * len(range(1, M, 3)) and not np.isnan(want).any()
    same_kinds(Y, want, "Y")
    fine = torch.from_numpy(np.isfinite(want)).cuda()
    assert torch.equal(Y[fine], Y0[fine])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 40, 300, 1600])
@pytest.mark.parametrize("where", [[("X", (1, 7), 1)], [("X", (1, 7), -1), ("X", (1, 71), 1)], [("A", (1, 3, 7), 1)],
                                   [("B", (1, 5, 3), 1)], [("dY", (1, 5), -1)]])
def test_an_infinity_in_the_backward(M, dtype, where):
    """dA is a sum of g x: infinite, with the formula's sign, where an infinity meets numbers; and dX and dB likewise."""
    c, d = one_infinity(M, dtype, where)
    Z = fwd(cuda(c))[1]
    first, got = bwd(cuda(c), Z), bwd(cuda(d), Z)
    with np.errstate(all="ignore"):
        want = O.multi_bwd(*(C.f64(d[k]) for k in ("X", "W0", "A", "B", "s")), c["ids"], C.f64(Z), C.f64(d["dY"]))
    for name, a, b, v in zip(("dX", "dA", "dB", "dbias"), first, got, want):
        same_kinds(b, v, name)
        fine = torch.from_numpy(np.isfinite(v)).cuda()
        assert torch.equal(a[fine], b[fine]), name


@pytest.mark.parametrize("e", [10, 40])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_products_that_overflow(M, sign, e):
    """Finite factors, z or g of 2^50 or 2^80, whose product does not fit in fp32, let alone bf16: the infinity of its
    sign, as one product of the rounded factor gives, whatever the sign of its rounding's rest."""
    for frac in (1 + 3 * 2.0 ** -7, 1 + 100 * 2.0 ** -7, 1):         # times 1 + 2^-7: rests of both signs and none
        c = C.inputs(M, 64, 72, 8, 2, "one", "bf16", bias=False)
        for k in ("A", "B", "W0", "X", "dY"):
            c[k][:] = 0
        c["s"][:] = 1
        c["A"][1, 3, 5], c["X"][:, 5], c["B"][1, 9, 3] = 2.0 ** e * (1 + 2.0 ** -7), 2.0 ** 40 * frac, sign * 2.0 ** (120 - e)
        g = cuda(c)
        Y, Z = fwd(g)
        assert (Y[:, 9] == sign * float("inf")).all() and not Y[:, :9].any() and not Y[:, 10:].any()
        g["dY"][0, 9], g["X"][0, 5], g["A"][:] = 2.0 ** (2 * e - 80) * frac, 2.0 ** (120 - e), 0
        g["s"][1] = 1 + 2.0 ** -7                        # g_0 = sign 2^(40 + e) (1 + 2^-7) frac
        dX, dA, dB, _ = bwd(g, torch.zeros_like(Z))
        assert dA[1, 3, 5] == sign * float("inf")
        dA[1, 3, 5] = 0
        assert not dA.any() and not dB.any() and not dX.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,r", [(40, 16), (300, 24), (1600, 72)])
def test_adapters_without_rows_have_zero_gradients(M, r, dtype):
    """Whatever their slots hold: scales, factors.  The others' bits are as with numbers there."""
    c = C.inputs(M, 136, 264, r, 5, "rows", dtype)
    c["ids"] = np.asarray([0, 2, -1, 4, 2])[np.arange(M) % 5]        # 1 and 3 have none
    g = cuda(c)
    Y0, Z0 = fwd(g)
    first = bwd(g, Z0)
    for k in ("A", "B", "s"):
        g[k][1], g[k][3] = float("nan"), float("inf")
    Y, Z = fwd(g)
    assert torch.equal(Y, Y0) and torch.equal(Z, Z0)
    for a, b in zip(first, bwd(g, Z)):
        assert torch.equal(a, b)
    for t in first[1:3]:
        assert not t[1].any() and not t[3].any() and t[[0, 2, 4]].any(-1).any(-1).all()


@pytest.mark.parametrize("M,r", [(40, 13), (300, 16), (600, 72)])
def test_what_is_not_finite_stays_with_its_adapter_in_fp32(M, r):
    c = C.inputs(M, 136, 264, r, 4, "rows", "f32")
    g = cuda(c)
    plan = ops.adapter_plan(g["ids"], 4)
    Y0, Z0 = fwd(g, plan)
    d0 = bwd(g, Z0, plan)
    g2 = {k: v.clone() if torch.is_tensor(v) else v for k, v in g.items()}
    g2["A"][1, :, ::3], g2["B"][1, ::2], g2["s"][1] = float("nan"), float("inf"), float("nan")
    sick = int(np.flatnonzero(c["ids"] == 2)[1])
    g2["X"][sick], g2["dY"][sick] = float("inf"), float("nan")
    Y, Z = fwd(g2, plan)
    fine = torch.from_numpy(c["ids"] != 1).cuda()
    fine[sick] = False
    assert torch.equal(Y[fine], Y0[fine]) and torch.equal(Z[fine], Z0[fine])
    dX, dA, dB, _ = bwd(g2, torch.where(fine[:, None], Z0, float("nan")), plan)
    assert torch.equal(dX[fine], d0[0][fine])
    for a in (0, 3):
        assert torch.equal(dA[a], d0[1][a]) and torch.equal(dB[a], d0[2][a])


@pytest.mark.parametrize("rows", [1000, 65536 + 37])
def test_fp32_gradients_of_many_rows(rows):
    """One adapter's rows are summed in shares: a sum whose every step would round down by almost half a step
    is off by the roundings of a share and of the shares' sum, not by one for each row.  Steps of a thread: 128 in
    a share, one for each 1024 rows; then 7 for the warps and one for the scale."""
    n, d, low = 3, 8, 1 + 0.98 * 2.0 ** -12
    v = float(np.float32(low))
    g = {"X": torch.full((rows, d), v), "W0": torch.zeros(d, d), "A": torch.zeros(n, 2, d), "B": torch.zeros(n, d, 2),
         "s": torch.ones(n), "dY": torch.ones(rows, d), "ids": torch.ones(rows, dtype=torch.int64)}
    g["B"][1, 0, 0] = g["B"][1, 3, 1] = 1                # g of both is one
    g = {k: t.cuda() for k, t in g.items()}
    Z = torch.full((rows, 2), v, device="cuda")
    dX, dA, dB, db = bwd(g, Z)
    off = (128 + rows // 1024 + 1 + 8) * 2.0 ** -24 * rows * v
    assert abs(C.f64(dA[1]) - rows * v).max() <= off
    assert abs(C.f64(dB[1]) - rows * v).max() <= off
    assert not dA[[0, 2]].any() and not dB[[0, 2]].any() and (db == rows).all()


@pytest.mark.parametrize("M", [3, 16, 40, 90, 250])
def test_recomputed_z_of_a_few_rows(M):
    """The forward of a few rows sums z in another order than the backward that recomputes it, which then has its own
    half step: the gradients meet the bound of z as the formula has it, off by that half step."""
    c = C.inputs(M, 136, 72, 16, 4, "rows", "bf16")
    g = cuda(c)
    X, W0, A, B, s, dY = (C.f64(c[k]) for k in ("X", "W0", "A", "B", "s", "dY"))
    Z = O.multi_fwd(X, W0, A, B, s, c["ids"])[1]
    mZ = O.multi_fwd(abs(X), W0, abs(A), B, s, c["ids"])[1]
    zero = np.zeros((M, 136))
    off_z = C.half_step("bf16") * abs(Z) + (136 + 4) * C.STEP * mZ * (1 + C.half_step("bf16"))
    more = O.multi_bwd(zero, W0, A, B, abs(s), c["ids"], off_z, abs(dY))[2]
    ref = C.reference_bwd(c, torch.from_numpy(Z), "bf16")
    ref["dB"] = (ref["dB"][0], ref["dB"][1] + more * (1 + 2 * C.half_step("bf16")))
    for k, v in zip(("dX", "dA", "dB", "dbias"), bwd(g, None)):
        C.near(v, ref[k], k)


@pytest.mark.parametrize("one_stream", [False, True])
def test_every_thread_comes_to_its_end(one_stream):
    """As test_threads; what a thread raises counts, and each has to finish its rounds."""
    cases = [cuda(C.inputs(M, d, d + 16, r, 5, "rows", dtype, seed=M)) for M, d, r, dtype in
             ((3, 520, 16, "bf16"), (90, 136, 24, "f32"), (400, 264, 72, "bf16"), (2570, 1800, 32, "bf16"))]
    plans = [ops.adapter_plan(g["ids"], 5) for g in cases]

    def step(i):
        Y, Z = fwd(cases[i], plans[i])
        grads = bwd(cases[i], Z, plans[i])
        return (Y, Z, optim.clip_grads([grads[1], grads[2]], 1.0, groups=5)) + grads

    want = [step(i) for i in range(4)]
    torch.cuda.synchronize()
    said = [None] * 4

    def run(i):
        try:
            stream = torch.cuda.default_stream() if one_stream else torch.cuda.Stream()
            rounds = 0
            with torch.cuda.stream(stream):
                for _ in range(20):
                    got = step(i)
                    stream.synchronize()
                    rounds += all(torch.equal(a, b) for a, b in zip(got, want[i]))
            said[i] = rounds
        except BaseException as e:  # noqa: BLE001
            said[i] = e

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert said == [20] * 4
    ops.check_device_errors()


@pytest.mark.parametrize("s", [float("nan"), float("inf"), -float("inf"), 1e39])
def test_a_scale_that_is_not_finite_in_fp32_is_named(s):
    """As it is without a GPU: a ValueError, before anything is launched."""
    g = cuda(C.inputs(8, 64, 72, 8, 3, "rows", "bf16"))
    plan, args = ops.adapter_plan(g["ids"], 3), (g["X"], g["W0"], g["A"], g["B"])
    with pytest.raises(ValueError, match="s must be finite"):
        ops.lora_multi_fwd(*args, s, plan)
    with pytest.raises(ValueError, match="s must be finite"):
        ops.lora_multi_bwd(*args, None, g["dY"], s, plan)
