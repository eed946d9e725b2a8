"""Cases of the operators around the adapted projections: the norms before and after a block with its
gate and residual scale, rotary positions, and the AdamW step over an adapter set.

`run` computes a case in plain torch operations in 32 bits, or (own = True) through the package."""
import math

import torch

own = False
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 256     # elements that share one scale of an 8-bit optimiser state


# ------------------------------------------------------------------ cases
def _norm(name, way, M, D, dtype, post, gate, alpha=1.0, offset=0.0):
    """way: fwd or bwd; post: a norm on the block's output; gate: none, row (one for all tokens), seq
    (one for each run of M / 4 tokens) or token."""
    return {"name": name, "op": "norm", "way": way, "M": M, "D": D, "dtype": dtype, "post": post, "gate": gate,
            "alpha": alpha, "offset": offset}


def _rotary(name, way, M, H, hd, rot, dtype, layout, scaling, packed, longest):
    """packed: H heads at the start of a row that holds H + H // 5 of them (query and key heads of a
    fused projection, the value heads left alone), rotated in place; otherwise a new tensor.
    longest: positions lie below it."""
    return {"name": name, "op": "rotary", "way": way, "M": M, "H": H, "hd": hd, "rot": rot, "dtype": dtype,
            "layout": layout, "scaling": scaling, "packed": packed, "longest": longest}


def _adamw(name, layers, rank, hidden, kv, inner, dtype, bits, clip):
    """The A and B of the seven projections of `layers` blocks."""
    return {"name": name, "op": "adamw", "layers": layers, "rank": rank, "hidden": hidden, "kv": kv, "inner": inner,
            "dtype": dtype, "bits": bits, "clip": clip}


def listed():
    return [
        # one token of a decode step between two blocks: latency
        _norm("norm_fwd_token", "fwd", 1, 4096, "bf16", True, "none"),
        # fp32 activations with a learned gate per channel, an uneven number of rows and columns
        _norm("norm_fwd_f32_509x1000", "fwd", 509, 1000, "f32", False, "row", 0.5),
        # the training workloads' token count and hidden size, norms on both sides of the block
        _norm("norm_fwd_16384x4096", "fwd", 16384, 4096, "bf16", True, "none", 1.0, 1.0),
        # a ragged batch of a smaller model, every token with its own gate
        _norm("norm_bwd_3001x2568", "bwd", 3001, 2568, "bf16", True, "token", 0.22),
        # its backward at full size with a gate for each sequence, all weight gradients
        _norm("norm_bwd_16384x4096", "bwd", 16384, 4096, "bf16", True, "seq"),
        # a decode step of 64 sequences far into a long context: latency
        _rotary("rotary_decode_64", "fwd", 64, 40, 128, 128, "bf16", "half", "bands", True, 131072),
        # part of an 80-wide head, adjacent pairs, fp32, an odd number of tokens
        _rotary("rotary_partial_f32", "fwd", 1999, 12, 80, 32, "f32", "interleaved", "linear", False, 8192),
        # query and key heads (32 + 8) of the training workload, positions scaled for a longer context
        _rotary("rotary_fwd_16384x40", "fwd", 16384, 40, 128, 128, "bf16", "half", "yarn", False, 65536),
        # its gradient, in place in the packed gradient of the projection, adjacent pairs
        _rotary("rotary_bwd_16384x40", "bwd", 16384, 40, 128, 128, "bf16", "interleaved", "none", True, 4096),
        # one fp32 block of a small model: 14 tensors, latency
        _adamw("adamw_f32_1_layer", 1, 8, 512, 128, 1376, "f32", 32, 0.0),
        # the adapters of 32 blocks (448 tensors), bf16 with fp32 masters, gradients clipped
        _adamw("adamw_bf16_32_layers", 32, 16, 4096, 1024, 14336, "bf16", 32, 1.0),
        # the same at rank 64 with 8-bit states
        _adamw("adamw8_bf16_32_layers", 32, 64, 4096, 1024, 14336, "bf16", 8, 0.0),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + (n == 3072)


def draw(rng):
    op = rng.choice(("norm", "norm", "rotary", "rotary", "adamw"))
    if op == "norm":
        D = 8 * _log(rng, 8, 1024)
        D += 8 * (D == 3072)
        M = _log(rng, 1, min(16384, 16384 * 4096 // D))
        gate = rng.choice(("none", "row", "seq", "token"))
        c = _norm("", rng.choice(("fwd", "bwd")), M + (-M) % 4 if gate == "seq" else M, D,
                  rng.choice(("bf16", "bf16", "f32")) if M * D <= 8192 * 4096 else "bf16",
                  rng.random() < 0.5, gate, rng.choice((1.0, 0.22, 0.5)), rng.choice((0.0, 1.0)))
    elif op == "rotary":
        hd = rng.choice((64, 72, 80, 96, 128, 256))
        rot = rng.choice((hd, hd, hd // 2, hd // 4))
        H = _log(rng, 1, 64)
        M = _log(rng, 1, min(16384, 16384 * 40 * 128 // (H * hd * 2)))
        way, scaling = rng.choice(("fwd", "bwd")), rng.choice(("none", "linear", "ntk", "bands", "yarn"))
        c = _rotary("", way, M, H, hd, rot, rng.choice(("bf16", "bf16", "f32")), rng.choice(("half", "interleaved")),
                    scaling, scaling != "yarn" and rng.random() < 0.5, _log(rng, 512, 131072))
    else:
        hidden = 64 * _log(rng, 4, 64)
        hidden += 64 * (hidden == 3072)
        kv = hidden // rng.choice((1, 4, 8))
        inner = hidden * rng.choice((11, 14, 16)) // 4
        inner += 8 * (inner == 3072)
        c = _adamw("", _log(rng, 1, 32), 8 * _log(rng, 1, 4), hidden, kv + 8 * (kv == 3072), inner,
                   rng.choice(("bf16", "bf16", "f32")), rng.choice((8, 32)), rng.choice((0.0, 1.0)))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _shapes(c):
    """(shape, step size factor, weight decay) of each tensor: A [r, n_in] and B [n_out, r] of the seven
    projections; B with a larger step and no decay."""
    h, k, i, r = c["hidden"], c["kv"], c["inner"], c["rank"]
    block = [(h, h), (k, h), (k, h), (h, h), (i, h), (i, h), (h, i)]
    return [t for _ in range(c["layers"]) for o, n in block
            for t in (((r, n), 1.0, 0.01), ((o, r), 4.0, 0.0))]


def _inv_freq(c):
    """Angle per position of each pair, float64, and the factor on the rotated values."""
    d, base, far, factor = c["rot"], 10000.0, 8192.0, 8.0
    i = torch.arange(d // 2, dtype=torch.float64, device=DEV)
    kind = c["scaling"]
    if kind == "ntk":
        base *= factor ** (d / max(d - 2, 1))
    f = base ** (-2 * i / d)
    if kind == "linear":
        f = f / factor
    elif kind == "bands":       # long waves stretched, short ones kept, a blend between
        low, high = 1.0, 4.0
        turns = far * f / (2 * math.pi)
        s = ((turns - low) / (high - low)).clamp(0, 1)
        f = (1 - s) * f / factor + s * f
    elif kind == "yarn":        # the same by the pair's index
        at = [d * math.log(far / (b * 2 * math.pi)) / (2 * math.log(base)) for b in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
        ramp = ((i - low) / (high - low if high > low else 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
    return f, 0.1 * math.log(factor) + 1 if kind == "yarn" else 1.0


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, scale=1.0, mean=0.0, dtype=dt):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(scale).add_(mean).to(dtype)

    s = {"case": c}
    if c["op"] == "norm":
        M, D, mean = c["M"], c["D"], 1.0 - c["offset"]
        rows = {"none": 0, "row": 1, "seq": min(4, M), "token": M}[c["gate"]]
        s["x"], s["y"] = normal(M, D, scale=2.0), normal(M, D)
        s["w_pre"] = normal(D, scale=0.1, mean=mean)
        s["w_post"] = normal(D, scale=0.1, mean=mean) if c["post"] else None
        s["gate"] = normal(rows, D, scale=0.5) if rows else None
        if c["way"] == "bwd":       # x stands for the block's output stream; the forward's row factors
            s["r_pre"] = torch.rsqrt(s["x"].float().square().mean(1) + 1e-6)
            s["r_post"] = torch.rsqrt(s["y"].float().square().mean(1) + 1e-6) if c["post"] else None
            s["dh"], s["dx"] = normal(M, D), normal(M, D)
    elif c["op"] == "rotary":
        M, H, hd = c["M"], c["H"], c["hd"]
        s["X"] = normal(M, (H + H // 5 if c["packed"] else H) * hd)
        s["pos"] = torch.randint(0, c["longest"], (M,), generator=gen, device=DEV)
        freq, s["scale"] = _inv_freq(c)
        angle = torch.arange(c["longest"], dtype=torch.float64, device=DEV)[:, None] * freq
        s["cos"], s["sin"] = (angle.cos() * s["scale"]).float(), (angle.sin() * s["scale"]).float()
        if own:
            from dora_adapter_linear_gb300 import ops
            s["plan"] = ops.rotary_plan(c["rot"], layout=c["layout"], inv_freq=freq, scale=s["scale"], device=DEV)
    else:
        shapes = _shapes(c)
        blocks = [-(-sh[0] * sh[1] // BLOCK) for sh, _, _ in shapes]
        nb = sum(blocks)
        count = torch.tensor(blocks, device=DEV)
        per = torch.tensor([(a, b) for _, a, b in shapes], device=DEV).repeat_interleave(count, 0)
        s["lr_mul"], s["decay"] = per[:, :1].contiguous(), per[:, 1:].contiguous()
        size = torch.tensor([sh[0] * sh[1] for sh, _, _ in shapes], device=DEV).repeat_interleave(count)
        first = (count.cumsum(0) - count).repeat_interleave(count)
        left = size - (torch.arange(nb, device=DEV) - first) * BLOCK
        real = torch.arange(BLOCK, device=DEV) < left[:, None]       # False in the padding of a last block
        # gradients of uneven size: a factor for each block of the state and one for each of its columns
        span = torch.exp(torch.randn(nb, 1, generator=gen, device=DEV)) * torch.exp(torch.randn(1, BLOCK, generator=gen, device=DEV))
        s["G"] = (torch.randn(nb, BLOCK, generator=gen, device=DEV) * span * 1e-3 * real).to(dt)
        s["m"] = torch.randn(nb, BLOCK, generator=gen, device=DEV) * span * 3e-4 * real
        s["v"] = (torch.rand(nb, BLOCK, generator=gen, device=DEV) + 0.5) * span.square() * 1e-6 * real
        master = torch.randn(nb, BLOCK, generator=gen, device=DEV) * 0.02 * real
        s["P"], s["master"] = master.to(dt), master if dt != torch.float32 else None
        if dt == torch.float32:
            s["P"] = master
        if c["bits"] == 8:
            s["m"], s["m_scale"] = _encode(s["m"], False)
            s["v"], s["v_scale"] = _encode(s["v"].sqrt(), True)
        s["t"], s["lr"], s["betas"], s["eps"] = 100, 1e-3, (0.9, 0.999), 1e-8
        if own:
            from dora_adapter_linear_gb300 import optim
            at, views = 0, []
            for (sh, _, _), b in zip(shapes, blocks):
                views.append([s[k].view(-1)[at:at + sh[0] * sh[1]].view(sh) for k in "PG"])
                at += b * BLOCK
            s["grads"] = [g for _, g in views]
            o = s["opt"] = optim.AdamW([p for p, _ in views], lr=s["lr"], betas=s["betas"], eps=s["eps"],
                                       weight_decay=[d for _, _, d in shapes], lr_mul=[a for _, a, _ in shapes],
                                       state_bits=c["bits"])
            o.load_state_dict({"step": s["t"], **{k: s.get(k) for k in ("m", "v", "m_scale", "v_scale", "master")}})
            for k in ("m", "v", "m_scale", "v_scale", "master"):
                s.pop(k, None)
    return s


# ------------------------------------------------------------------ plain forms
def _encode(x, magnitude):
    """8-bit floating codes (4 exponent, 3 mantissa bits) of each row and its scale; a magnitude above
    zero keeps the smallest code."""
    top = x.abs().amax(1, keepdim=True)
    code = (x * torch.where(top > 0, 448.0 / top, 0.0)).clamp(-448.0, 448.0)
    if magnitude:
        code = torch.where(x > 0, code.clamp_min(2.0 ** -9), code)
    return code.to(torch.float8_e4m3fn), top / 448.0


def _plain_norm(s):
    c = s["case"]
    M, D = c["M"], c["D"]
    x, y, off = s["x"].float(), s["y"].float(), c["offset"]
    wz = s["w_pre"].float() + off
    wp = s["w_post"].float() + off if c["post"] else None
    g = s["gate"].float().repeat_interleave(M // s["gate"].shape[0], 0) if s["gate"] is not None else None
    dt = s["x"].dtype
    if c["way"] == "fwd":
        r_y = torch.rsqrt(y.square().mean(1) + 1e-6) if c["post"] else None
        p = y * r_y[:, None] * wp if c["post"] else y
        z = x + c["alpha"] * (p * g if g is not None else p)
        r_z = torch.rsqrt(z.square().mean(1) + 1e-6)
        return z.to(dt), (z * r_z[:, None] * wz).to(dt), r_z, r_y
    dh, r_z = s["dh"].float(), s["r_pre"][:, None]
    wdh = wz * dh
    dz = s["dx"].float() + r_z * (wdh - x * r_z.square() * (wdh * x).mean(1, keepdim=True))
    dw_pre = (dh * x * r_z).sum(0).to(dt)
    dp = c["alpha"] * (dz * g if g is not None else dz)
    p, dy, dw_post = y, dp, None
    if c["post"]:
        r_y = s["r_post"][:, None]
        n = y * r_y
        p, wdp = n * wp, wp * dp
        dy = r_y * (wdp - n * (wdp * n).mean(1, keepdim=True))
        dw_post = (dp * n).sum(0).to(dt)
    dg = (c["alpha"] * dz * p).view(s["gate"].shape[0], -1, D).sum(1).to(dt) if g is not None else None
    return dz.to(dt), dy.to(dt), dw_pre, dw_post, dg


def _plain_rotary(s):
    c = s["case"]
    M, H, hd, rot = c["M"], c["H"], c["hd"], c["rot"]
    X = s["X"][:, :H * hd].view(M, H, hd)
    x = X[..., :rot].float()
    half = c["layout"] == "half"
    a, b = (x[..., :rot // 2], x[..., rot // 2:]) if half else (x[..., 0::2], x[..., 1::2])
    cos, sin = s["cos"][s["pos"]][:, None], s["sin"][s["pos"]][:, None]
    if c["way"] == "bwd":
        sin = -sin
    a, b = a * cos - b * sin, b * cos + a * sin
    r = (torch.cat((a, b), -1) if half else torch.stack((a, b), -1).flatten(-2)).to(X.dtype)
    if c["packed"]:
        X[..., :rot] = r
        return s["X"]
    return torch.cat((r, X[..., rot:]), -1)


def _plain_adamw(s):
    c = s["case"]
    b1, b2 = s["betas"]
    s["t"] += 1
    g, norm = s["G"].float(), None
    if c["clip"]:
        norm = g.square().sum().sqrt()
        g = g * (c["clip"] / (norm + 1e-6)).clamp(max=1.0)
    if c["bits"] == 8:
        m = s["m"].float() * s["m_scale"]
        v = (s["v"].float() * s["v_scale"]).square()
    else:
        m, v = s["m"], s["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    lr = s["lr"] * s["lr_mul"]
    p = s["P"] if s["master"] is None else s["master"]
    step = (m / (1 - b1 ** s["t"])) / ((v / (1 - b2 ** s["t"])).sqrt() + s["eps"])
    p.copy_(p - lr * s["decay"] * p - lr * step)
    if s["master"] is not None:
        s["P"].copy_(p)
    if c["bits"] == 8:
        s["m"], s["m_scale"] = _encode(m, False)
        s["v"], s["v_scale"] = _encode(v.sqrt(), True)
    else:
        s["m"], s["v"] = m, v
    return s["P"], s["master"], s["m"], s["v"], s.get("m_scale"), s.get("v_scale"), norm


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"norm": _plain_norm, "rotary": _plain_rotary, "adamw": _plain_adamw}[c["op"]](s)
    from dora_adapter_linear_gb300 import ops
    if c["op"] == "norm":
        how = dict(w_pre=s["w_pre"], w_post=s["w_post"], gate=s["gate"], post_norm=c["post"], alpha=c["alpha"],
                   w_offset=c["offset"])
        if c["way"] == "fwd":
            return ops.block_norm_fwd(s["x"], s["y"], eps=1e-6, **how)
        return ops.block_norm_bwd(s["x"], s["y"], s["r_pre"], s["r_post"], s["dh"], s["dx"], **how)
    if c["op"] == "rotary":
        X = s["X"][:, :c["H"] * c["hd"]].view(c["M"], c["H"], c["hd"])
        Y = (ops.rotary_fwd if c["way"] == "fwd" else ops.rotary_bwd)(X, s["pos"], s["plan"],
                                                                      out=X if c["packed"] else None)
        return s["X"] if c["packed"] else Y
    o = s["opt"]
    norm = o.step(s["grads"], max_norm=c["clip"] or None)
    return s["P"], o.master, o.m, o.v, o.m_scale, o.v_scale, norm


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        M, D = c["M"], c["D"]
        rows = {"none": 0, "row": 1, "seq": min(4, M), "token": M}[c["gate"]]
        w = 1 + c["post"]
        if c["way"] == "fwd":
            return {"bytes": e * D * (4 * M + w + rows) + 4 * M * w, "flops": 10 * M * D}
        return {"bytes": e * D * (6 * M + 2 * w + 2 * rows) + 4 * M * w, "flops": 24 * M * D}
    if c["op"] == "rotary":
        n = c["M"] * c["H"]
        return {"bytes": 2 * e * n * (c["rot"] if c["packed"] else c["hd"]) + 8 * c["M"], "flops": 3 * n * c["rot"]}
    n = sum(sh[0] * sh[1] for sh, _, _ in _shapes(c))
    param = e + 8 if e == 2 else 8                      # bf16 written, master read and written; fp32 both ways
    state = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * (e + param + state), "flops": 16 * n}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s, c = prepare(case, seed), case
    f64 = lambda t: None if t is None else t.to(torch.float64)  # noqa: E731
    if c["op"] == "norm":
        M, D, alpha = c["M"], c["D"], c["alpha"]
        x, y = f64(s["x"]), f64(s["y"])
        w = f64(s["w_pre"]) + c["offset"]
        u = f64(s["w_post"]) + c["offset"] if c["post"] else torch.ones(D, dtype=torch.float64, device=DEV)
        gate = s["gate"]
        gsel = torch.arange(M, device=DEV) // (M // gate.shape[0]) if gate is not None else None
        g = f64(gate)[gsel] if gate is not None else torch.ones((), dtype=torch.float64, device=DEV)
        ry = (y.pow(2).mean(1, True) + 1e-6).pow(-0.5) if c["post"] else torch.ones(M, 1, dtype=torch.float64, device=DEV)
        if c["way"] == "fwd":
            z = x + alpha * g * u * y * ry
            rz = (z.pow(2).mean(1, True) + 1e-6).pow(-0.5)
            return z, z * rz * w, rz[:, 0], ry[:, 0] if c["post"] else None
        dh = f64(s["dh"])
        rz = (x.pow(2).mean(1, True) + 1e-6).pow(-0.5)
        a = dh * w
        dz = f64(s["dx"]) + rz * a - x * rz.pow(3) * (a * x).sum(1, True) / D
        b = alpha * g * dz                              # gradient of the normed block output
        dy = b
        if c["post"]:
            dy = ry * b * u - y * ry.pow(3) * (b * u * y).sum(1, True) / D
        dg = None
        if gate is not None:
            dg = torch.zeros_like(gate, dtype=torch.float64).index_add_(0, gsel, alpha * dz * y * ry * u)
        return dz, dy, (dh * x * rz).sum(0), (b * y * ry).sum(0) if c["post"] else None, dg
    if c["op"] == "rotary":
        n, H, hd, rot = c["M"], c["H"], c["hd"], c["rot"]
        whole = f64(s["X"])
        X = whole[:, :H * hd].reshape(n, H, hd)
        f, scale = _inv_freq(c)
        t = s["pos"].double()[:, None, None] * f * (1.0 if c["way"] == "fwd" else -1.0)
        turn = torch.polar(torch.full_like(t, scale), t)
        pairs = X[..., :rot].reshape(n, H, 2, rot // 2).transpose(-1, -2) if c["layout"] == "half" else \
            X[..., :rot].reshape(n, H, rot // 2, 2)
        r = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        r = (r.transpose(-1, -2) if c["layout"] == "half" else r).reshape(n, H, rot)
        Y = torch.cat((r, X[..., rot:]), -1)
        return torch.cat((Y.reshape(n, H * hd), whole[:, H * hd:]), 1) if c["packed"] else Y
    b1, b2 = s["betas"]
    t = s["t"] + 1
    g, norm = f64(s["G"]), None
    if c["clip"]:
        norm = g.pow(2).sum().sqrt()
        g = g * min(1.0, c["clip"] / (float(norm) + 1e-6))
    m, v = f64(s["m"]), f64(s["v"])
    if c["bits"] == 8:
        m, v = m * f64(s["m_scale"]), (v * f64(s["v_scale"])).pow(2)
    m, v = m.mul_(b1).add_(g, alpha=1 - b1), v.mul_(b2).addcmul_(g, g, value=1 - b2)
    del g
    p = f64(s["P"] if s["master"] is None else s["master"])
    lr = s["lr"] * f64(s["lr_mul"])
    p = p * (1 - lr * f64(s["decay"])) - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + s["eps"])
    master = None if s["master"] is None else p
    if c["bits"] == 32:
        return p, master, m, v, None, None, norm
    out = []
    for x, low in ((m, 0.0), (v.sqrt_(), 2.0 ** -9)):
        top = x.abs().amax(1, keepdim=True)
        q = x / top.clamp_min(1e-300) * 448.0
        out.append((torch.where(q > 0, q.clamp_min(low), q), top / 448.0))      # before the rounding to a code
    return p, master, out[0][0], out[1][0], out[0][1], out[1][1], norm
