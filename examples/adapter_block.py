"""Fine-tunes the adapters of one transformer block with the library's calls, then decodes with it.

The block: norm - fused query/key/value projection - rotary positions - attention - output projection -
norm with gate and residual - gated MLP - norm with gate and residual.  Its weights are frozen; the A and
B of its seven adapters learn to imitate a block with other adapters.  Attention itself is plain torch.

    python examples/adapter_block.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from dora_adapter_linear_gb300 import ops, optim  # noqa: E402


class Block:
    def __init__(self, hidden=512, heads=8, kv_heads=2, head_dim=64, inner=1408, rank=8, seed=0, device="cuda"):
        self.heads, self.kv_heads, self.head_dim, self.s = heads, kv_heads, head_dim, 2.0
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen, device=device) * scale).bfloat16()

        self.nq, self.nk = heads * head_dim, kv_heads * head_dim
        sizes = {"q": (self.nq, hidden), "k": (self.nk, hidden), "v": (self.nk, hidden), "o": (hidden, self.nq),
                 "g": (inner, hidden), "u": (inner, hidden), "d": (hidden, inner)}
        self.W = {n: normal(o, i, scale=i ** -0.5) for n, (o, i) in sizes.items()}
        self.W["qkv"] = torch.cat([self.W.pop(n) for n in "qkv"])
        self.A = {n: normal(rank, i, scale=i ** -0.5) for n, (_, i) in sizes.items()}
        self.B = {n: normal(o, rank, scale=0.0) for n, (o, _) in sizes.items()}
        self.norms = {n: normal(hidden, scale=0.1) + 1 for n in ("attn", "attn_post", "mlp", "mlp_post", "out")}
        self.gate = {n: normal(1, hidden, scale=0.1) + 1 for n in ("attn", "mlp")}
        self.plan = ops.rotary_plan(head_dim, base=500000.0, scaling="bands", factor=8.0, device=device)

    def adapters(self):
        """The trained tensors: A and B of q, k, v, o, g, u, d."""
        return [t for n in self.A for t in (self.A[n], self.B[n])]

    def _leaves(self):
        return [(self.A[n], self.B[n], self.s) for n in "qkv"]

    def _proj(self, n):
        return {"W": self.W[n], "A": self.A[n], "B": self.B[n], "s": self.s}

    def _post(self, part):
        return dict(w_post=self.norms[part + "_post"], gate=self.gate[part], post_norm=True, alpha=0.5)

    def forward(self, X, pos, batch, past=None):
        """X [batch * T, hidden], pos [batch * T].  past: (keys, values) [batch, kv_heads, before, head_dim] of
        earlier tokens.  Returns (output of the last norm, what the backward needs, keys and values so far)."""
        s = {"X0": X}
        _, s["H0"], s["r0"], _ = ops.block_norm_fwd(X, w_pre=self.norms["attn"])
        qkv, s["Zqkv"] = ops.lora_qkv_fwd(s["H0"], self.W["qkv"], self._leaves())
        turned = qkv[:, :self.nq + self.nk].view(X.shape[0], self.heads + self.kv_heads, self.head_dim)
        ops.rotary_fwd(turned, pos, self.plan, out=turned)      # queries and keys, in place
        s["qkv"] = qkv
        s["att"], kv = self._attention(qkv, batch, past)
        Y, s["Zo"] = ops.lora_linear_fwd(s["att"], self.W["o"], self.A["o"], self.B["o"], self.s)
        s["Y1"] = Y
        s["X1"], s["H1"], s["r1"], s["p1"] = ops.block_norm_fwd(X, Y, w_pre=self.norms["mlp"], **self._post("attn"))
        s["Y2"], s["mlp"] = ops.lora_mlp_swiglu_fwd(s["H1"], *map(self._proj, "gud"))
        s["X2"], out, s["r2"], s["p2"] = ops.block_norm_fwd(s["X1"], s["Y2"], w_pre=self.norms["out"],
                                                            **self._post("mlp"))
        return out, s, kv

    def _attention(self, qkv, batch, past=None):
        T, hd = qkv.shape[0] // batch, self.head_dim
        q, k, v = (t.view(batch, T, -1, hd).transpose(1, 2) for t in qkv.split([self.nq, self.nk, self.nk], 1))
        if past is not None:
            k, v = torch.cat((past[0], k), 2), torch.cat((past[1], v), 2)
        before = k.shape[2] - T
        kk, vv = (t.repeat_interleave(self.heads // self.kv_heads, 1).float() for t in (k, v))
        scores = q.float() @ kk.transpose(-1, -2) / math.sqrt(hd)
        seen = torch.arange(before + T, device=q.device) <= before + torch.arange(T, device=q.device)[:, None]
        out = torch.softmax(scores.masked_fill(~seen, float("-inf")), -1) @ vv
        return out.transpose(1, 2).reshape(batch * T, -1).to(qkv.dtype), (k, v)

    def backward(self, s, pos, batch, dOut):
        """Gradients of adapters() in their order, from the gradient of the output."""
        g = {}
        dX2, dY2, *_ = ops.block_norm_bwd(s["X2"], s["Y2"], s["r2"], s["p2"], dOut, None, w_pre=self.norms["out"],
                                          need_dw=False, need_dgate=False, **self._post("mlp"))
        m = ops.lora_mlp_swiglu_bwd(s["H1"], *map(self._proj, "gud"), s["mlp"], dY2)
        for n in "gud":
            g[n] = (m["dA" + n], m["dB" + n])
        dX1, dY1, *_ = ops.block_norm_bwd(s["X1"], s["Y1"], s["r1"], s["p1"], m["dX"], dX2, w_pre=self.norms["mlp"],
                                          need_dw=False, need_dgate=False, **self._post("attn"))
        datt, *g["o"], _ = ops.lora_linear_bwd(s["att"], self.W["o"], self.A["o"], self.B["o"], s["Zo"], dY1, self.s)
        qkv = s["qkv"].detach().requires_grad_(True)
        with torch.enable_grad():
            dqkv, = torch.autograd.grad(self._attention(qkv, batch)[0], qkv, datt)
        turned = dqkv[:, :self.nq + self.nk].view(dqkv.shape[0], self.heads + self.kv_heads, self.head_dim)
        ops.rotary_bwd(turned, pos, self.plan, out=turned)
        _, dA, dB, _ = ops.lora_qkv_bwd(s["H0"], self.W["qkv"], self._leaves(), s["Zqkv"], dqkv, need_dx=False)
        for i, n in enumerate("qkv"):
            g[n] = (dA[i], dB[i])
        return [t for n in self.A for t in g[n]]


def train(block, teacher, steps=60, batch=4, tokens=96, lr=2e-3, state_bits=8, seed=1):
    """Losses of `steps` AdamW steps: the mean squared distance to the teacher's output.  B takes four
    times A's step, without decay."""
    params = block.adapters()
    opt = optim.AdamW(params, lr=lr, weight_decay=[0.01, 0.0] * (len(params) // 2), lr_mul=[1.0, 4.0] * (len(params) // 2),
                      state_bits=state_bits)
    gen = torch.Generator(device=params[0].device).manual_seed(seed)
    pos = torch.arange(tokens, device=params[0].device).repeat(batch)
    losses = []
    for _ in range(steps):
        X = torch.randn(batch * tokens, block.W["o"].shape[0], generator=gen, device=pos.device).bfloat16()
        want = teacher.forward(X, pos, batch)[0].float()
        out, saved, _ = block.forward(X, pos, batch)
        off = out.float() - want
        losses.append(off.square().mean())
        dOut = (off * (2 / off.numel())).to(out.dtype)
        opt.step(block.backward(saved, pos, batch, dOut), max_norm=1.0)
    return torch.stack(losses).tolist()


def decode(block, X, batch):
    """The block's output for X [batch, T, hidden], one token of every sequence at a time."""
    out, past = [], None
    for t in range(X.shape[1]):
        pos = torch.full((batch,), t, device=X.device)
        o, _, past = block.forward(X[:, t].contiguous(), pos, batch, past)
        out.append(o)
    return torch.stack(out, 1)


def pair(**kw):
    """A block and a teacher of the same frozen weights whose adapters are not zero."""
    block, teacher = Block(**kw), Block(**kw)
    for i, n in enumerate(teacher.B):
        gen = torch.Generator(device=teacher.B[n].device).manual_seed(100 + i)
        teacher.B[n].copy_(torch.randn(teacher.B[n].shape, generator=gen, device=teacher.B[n].device) * 0.05)
    return block, teacher


if __name__ == "__main__":
    from dora_adapter_linear_gb300.build import build
    build()
    block, teacher = pair()
    losses = train(block, teacher, int(sys.argv[1]) if len(sys.argv) > 1 else 200)
    for i in range(0, len(losses), max(len(losses) // 10, 1)):
        print(f"step {i:4d}  loss {losses[i]:.5f}")
    print(f"last       loss {losses[-1]:.5f}")
    X = torch.randn(2, 24, 512, device="cuda").bfloat16()
    whole = block.forward(X.view(48, 512), torch.arange(24, device="cuda").repeat(2), 2)[0].view(2, 24, 512)
    print("token by token against the whole sequence, largest difference:", float((decode(block, X, 2) - whole).abs().max()))
