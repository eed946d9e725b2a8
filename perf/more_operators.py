"""Cases of the operators for many adapters beside one projection: the projection of a batch whose rows
have different adapters, its gradients, and the norms and clipping of many adapters' gradients.

`run` computes a case in plain torch operations in 32 bits, or (own = True) through the package."""
import math
import random

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def _multi(name, way, M, d_in, d_out, r, n, requests, dtype="bf16", bias=False, bare=False):
    """M rows of `requests` requests behind one another (M of them: every row its own), each with one of n
    adapters of rank r; bare: some requests have none.  bias: the projection has one (backward: its gradient)."""
    return {"name": name, "op": "multi", "way": way, "M": M, "d_in": d_in, "d_out": d_out, "r": r, "n": n,
            "requests": requests, "dtype": dtype, "bias": bias, "bare": bare}


def _clip(name, layers, rank, hidden, kv, inner, n, dtype, stacked):
    """The gradients of n adapters of the seven projections of `layers` blocks.  stacked: those of all adapters
    in one tensor, [n, ...]; otherwise each adapter's A and B are tensors of their own."""
    return {"name": name, "op": "clip", "layers": layers, "rank": rank, "hidden": hidden, "kv": kv, "inner": inner,
            "n": n, "dtype": dtype, "stacked": stacked}


def listed():
    return [
        # a decode step of one sequence: latency
        _multi("fwd_token", "fwd", 1, 4096, 4096, 16, 8, 1),
        # a decode step of 64 sequences, each with its own adapter out of 128
        _multi("fwd_decode_64", "fwd", 64, 4096, 4096, 16, 128, 64),
        # a decode step into the inner size of an MLP, an odd number of rows, high rank, some without adapter
        _multi("fwd_decode_19x11008", "fwd", 19, 4096, 11008, 64, 6, 19, bias=True, bare=True),
        # fp32, uneven sizes, a rank that is no multiple of 8
        _multi("fwd_f32_509x1000", "fwd", 509, 1000, 1496, 12, 5, 9, "f32", bias=True),
        # short prompts of many requests, more adapters than a tile has room for
        _multi("fwd_ragged_3001x2568", "fwd", 3001, 2568, 2568, 24, 37, 90, bare=True),
        # prompts of 16 requests at the projection of the headline workload
        _multi("fwd_prompts_8192x4096", "fwd", 8192, 4096, 4096, 16, 8, 16),
        # gradients of three small adapters in fp32
        _multi("bwd_f32_300x512", "bwd", 300, 512, 1376, 8, 3, 7, "f32"),
        # gradients of an uneven batch, with those of the bias, some sequences without adapter
        _multi("bwd_ragged_1999x1000", "bwd", 1999, 1000, 2568, 8, 11, 30, bias=True, bare=True),
        # eight adapters trained in one batch
        _multi("bwd_train_8192x11008", "bwd", 8192, 4096, 11008, 32, 8, 24),
        # clipping three adapters of one block of a small model: latency
        _clip("clip_f32_1_layer", 1, 8, 512, 128, 1376, 3, "f32", True),
        # one list of all adapters' tensors, uneven sizes
        _clip("clip_list_2_layers", 2, 24, 1000, 200, 2568, 5, "bf16", False),
        # the stacked gradients of four adapters of 32 blocks
        _clip("clip_bf16_32_layers", 32, 16, 4096, 1024, 14336, 4, "bf16", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.75:
        way = rng.choice(("fwd", "fwd", "bwd"))
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        d_in, d_out = 8 * _log(rng, 16, 512), 8 * _log(rng, 16, 1376)
        top = 8192 if dtype == "bf16" else 1024
        M = _log(rng, 1, 256) if rng.random() < 0.4 else _log(rng, 256, top)
        n = _log(rng, 1, 64)
        r = 8 * rng.choice((1, 2, 2, 3, 4)) if dtype == "bf16" else _log(rng, 1, 32)
        requests = M if M <= 256 and rng.random() < 0.7 else _log(rng, 1, max(1, min(M, 200)))
        c = _multi("", way, M, d_in, d_out, r, n, requests, dtype, rng.random() < 0.4, rng.random() < 0.4)
    else:
        hidden = 8 * _log(rng, 16, 512)
        c = _clip("", _log(rng, 1, 16), 8 * rng.choice((1, 2, 3)), hidden, 8 * max(1, hidden // 8 // rng.choice((1, 4, 8))),
                  8 * (hidden * rng.choice((11, 14, 16)) // 32), rng.choice((1, 2, 3, 5)), rng.choice(("bf16", "f32")),
                  rng.random() < 0.6)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _ids(c, seed):
    """The adapter of each row, -1 for none."""
    rng = random.Random(seed)
    M, req = c["M"], c["requests"]
    cuts = [0] + sorted(rng.sample(range(1, M), req - 1)) + [M]
    out = []
    for a, b in zip(cuts, cuts[1:]):
        out += [-1 if c["bare"] and rng.random() < 0.2 else rng.randrange(c["n"])] * (b - a)
    return out


def _shapes(c):
    h, k, i, r = c["hidden"], c["kv"], c["inner"], c["rank"]
    block = [(h, h), (k, h), (k, h), (h, h), (i, h), (i, h), (h, i)]
    return [t for _ in range(c["layers"]) for o, n in block for t in ((r, n), (o, r))]


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(scale).to(dt)

    s = {"case": c}
    if c["op"] == "clip":
        # one buffer, as a training program keeps them: for every tensor of the block the n adapters' behind one
        # another.  Every second adapter's gradients are far above the limit, the others below it.
        n, sizes = c["n"], [a * b for a, b in _shapes(c)]
        unit = math.gcd(*sizes)
        s["of"] = torch.tensor([g for z in sizes for g in range(n)], device=DEV).repeat_interleave(
            torch.tensor([z // unit for z in sizes for _ in range(n)], device=DEV))     # adapter of each `unit` elements
        size = torch.tensor([(10.0 if g % 2 == 0 else 0.2) / math.sqrt(sum(sizes)) for g in range(n)], device=DEV)
        flat = torch.randn(len(s["of"]), unit, generator=gen, device=DEV) * size[s["of"]][:, None]
        s["flat"], s["max_norm"] = flat.to(dt).view(-1), 1.0
        if own:
            parts = s["flat"].split([n * z for z in sizes])
            s["grads"], s["groups"] = [p.view(n, *sh) for p, sh in zip(parts, _shapes(c))], n
            if not c["stacked"]:
                s["grads"] = [t for stack in s["grads"] for t in stack]
                s["groups"] = [g for _ in sizes for g in range(n)]
        return s
    M, d_in, d_out, r, n = (c[k] for k in ("M", "d_in", "d_out", "r", "n"))
    s["ids"] = torch.tensor(_ids(c, seed), device=DEV)
    s["X"], s["W0"] = normal(M, d_in), normal(d_out, d_in, scale=d_in ** -0.5)
    s["A"], s["B"] = normal(n, r, d_in, scale=d_in ** -0.5), normal(n, d_out, r, scale=0.05)
    s["s"] = torch.rand(n, generator=gen, device=DEV) * 2 + 0.5
    s["bias"] = normal(d_out, scale=0.1) if c["bias"] else None
    if c["way"] == "bwd":
        s["dY"] = normal(M, d_out, scale=0.1)
        s["Z"] = _own_only(s, s["X"].float() @ s["A"].view(n * r, d_in).float().T).sum(1).to(dt)   # from the forward
    if own:
        from dora_adapter_linear_gb300 import ops
        s["plan"] = ops.adapter_plan(s["ids"], n)
    return s


# ------------------------------------------------------------------ plain forms
def _own_only(s, wide):
    """Products with all n adapters [M, n r], those of other adapters than the row's own set to zero."""
    n = s["A"].shape[0]
    mine = s["ids"][:, None] == torch.arange(n, device=DEV)
    return torch.where(mine[:, :, None], wide.view(len(s["ids"]), n, -1), 0.0)


def _plain_fwd(s):
    X, A, B, dt = s["X"].float(), s["A"], s["B"], s["X"].dtype
    n, r, d_in = A.shape
    Y = X @ s["W0"].float().T
    if X.shape[0] <= 256:       # a few rows: each with its own copy of its adapter
        at, some = s["ids"].clamp(min=0), (s["ids"] >= 0)[:, None]
        Z = torch.where(some, (A[at].float() @ X[:, :, None])[:, :, 0], 0.0)
        Y = Y + (B[at].float() @ (Z * s["s"][at][:, None])[:, :, None])[:, :, 0]
    else:
        wide = _own_only(s, X @ A.view(n * r, d_in).float().T)
        Z = wide.sum(1)
        Y = Y + (wide * s["s"][:, None]).flatten(1) @ B.float().transpose(1, 2).reshape(n * r, -1)
    if s["bias"] is not None:
        Y = Y + s["bias"].float()
    return Y.to(dt), Z.to(dt)


def _plain_bwd(s):
    X, dY, A, B, dt = s["X"].float(), s["dY"].float(), s["A"], s["B"], s["X"].dtype
    n, r, d_in = A.shape
    G = dY @ B.float().transpose(1, 2).reshape(n * r, -1).T
    G = (_own_only(s, G) * s["s"][:, None]).flatten(1)
    Z = _own_only(s, s["Z"].float().repeat(1, n)).flatten(1)
    dX = dY @ s["W0"].float() + G @ A.view(n * r, d_in).float()
    dA = (G.T @ X).view(n, r, d_in)
    dB = (Z.T @ dY).view(n, r, -1).transpose(1, 2) * s["s"][:, None, None]
    return dX.to(dt), dA.to(dt), dB.to(dt).contiguous(), dY.sum(0).to(dt) if s["bias"] is not None else None


def _plain_clip(s):
    g = s["flat"].view(len(s["of"]), -1).float()
    norm = torch.zeros(s["case"]["n"], dtype=torch.float64, device=DEV)
    norm = norm.index_add_(0, s["of"], g.square().sum(1).double()).sqrt().float()
    factor = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    s["flat"].copy_((g * factor[s["of"]][:, None]).view(-1))
    return norm, s["flat"]


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_clip(s) if c["op"] == "clip" else _plain_fwd(s) if c["way"] == "fwd" else _plain_bwd(s)
    from dora_adapter_linear_gb300 import ops, optim
    if c["op"] == "clip":
        return optim.clip_grads(s["grads"], s["max_norm"], groups=s["groups"]), s["flat"]
    if c["way"] == "fwd":
        return ops.lora_multi_fwd(s["X"], s["W0"], s["A"], s["B"], s["s"], s["plan"], bias=s["bias"])
    return ops.lora_multi_bwd(s["X"], s["W0"], s["A"], s["B"], s["Z"], s["dY"], s["s"], s["plan"],
                              need_dbias=c["bias"])


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "clip":
        each = sum(a * b for a, b in _shapes(c))
        scaled = (c["n"] + 1) // 2                      # adapters whose gradients are written
        return {"bytes": e * each * (c["n"] + scaled), "flops": each * (2 * c["n"] + scaled)}
    M, i, o, r, n = (c[k] for k in ("M", "d_in", "d_out", "r", "n"))
    used = min(n, c["requests"])                        # at most: the requests may share some
    if c["way"] == "fwd":
        return {"bytes": e * (M * (i + o + r) + o * i + used * r * (i + o)), "flops": 2 * M * (i * o + r * (i + o))}
    return {"bytes": e * (M * (2 * i + o + r) + o * i + (used + n) * r * (i + o)),
            "flops": 2 * M * (i * o + 2 * r * (i + o))}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    if c["op"] == "clip":
        stacks = f64(s["flat"]).split([c["n"] * a * b for a, b in _shapes(c)])
        norms = torch.stack([t.view(c["n"], -1).pow(2).sum(1) for t in stacks]).sum(0).sqrt()
        factors = [min(1.0, s["max_norm"] / (v + 1e-6)) for v in norms.tolist()]
        return norms, torch.cat([t * f for stack in stacks for t, f in zip(stack.view(c["n"], -1), factors)])
    M, n = c["M"], c["n"]
    X, W, A, B = f64(s["X"]), f64(s["W0"]), f64(s["A"]), f64(s["B"])
    scale = f64(s["s"])
    mine = [s["ids"] == a for a in range(n)]            # a row of truth values for each adapter
    if c["way"] == "fwd":
        Y, Z = torch.matmul(X, W.t()), torch.zeros(M, c["r"], dtype=torch.float64, device=DEV)
        for a in range(n):
            Z[mine[a]] = torch.matmul(X[mine[a]], A[a].t())
            Y[mine[a]] += scale[a] * torch.matmul(Z[mine[a]], B[a].t())
        return (Y if s["bias"] is None else Y + f64(s["bias"])), Z
    dY, Z = f64(s["dY"]), f64(s["Z"])
    dX = torch.matmul(dY, W)
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for a in range(n):
        G = scale[a] * torch.matmul(dY[mine[a]], B[a])
        dX[mine[a]] += torch.matmul(G, A[a])
        dA[a] = torch.matmul(G.t(), X[mine[a]])
        dB[a] = scale[a] * torch.matmul(dY[mine[a]].t(), Z[mine[a]])
    return dX, dA, dB, dY.sum(0) if s["bias"] is not None else None
