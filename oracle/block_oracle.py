"""Plain fp64 reference of the operators around the adapted projections: block norm, rotary positions
and AdamW.  Like lora_oracle it shares no code with the CUDA path."""
import numpy as np


def _rows(gate, M, rows_per_gate):
    return np.ones((M, 1)) if gate is None else gate[np.arange(M) // rows_per_gate]


def block_norm_fwd(x, y=None, w_pre=None, w_post=None, gate=None, rows_per_gate=1, alpha=1.0, eps=1e-6, off=0.0,
                   post=False):
    """(z, h, r_pre, r_post): z = x + alpha gate o p, p = y or its RMS norm, h the RMS norm of z."""
    z, r_post = x, None
    if y is not None:
        p = y
        if post:
            r_post = 1.0 / np.sqrt((y ** 2).mean(1) + eps)
            p = y * r_post[:, None] * (1.0 if w_post is None else w_post + off)
        z = x + alpha * _rows(gate, x.shape[0], rows_per_gate) * p
    r_pre = 1.0 / np.sqrt((z ** 2).mean(1) + eps)
    return z, z * r_pre[:, None] * (1.0 if w_pre is None else w_pre + off), r_pre, r_post


def block_norm_bwd(z, y, r_pre, r_post, dh, dz_in, w_pre=None, w_post=None, gate=None, rows_per_gate=1, alpha=1.0,
                   off=0.0, post=False):
    """(dx, dy, dw_pre, dw_post, dgate) from the gradients of h and z (either may be None)."""
    M, D = z.shape
    dz = np.zeros_like(z) if dz_in is None else dz_in.copy()
    dw_pre = np.zeros(D)
    if dh is not None:
        n = z * r_pre[:, None]
        a = dh * (1.0 if w_pre is None else w_pre + off)
        dz += r_pre[:, None] * (a - n * (a * n).mean(1, keepdims=True))
        dw_pre = (dh * n).sum(0)
    if y is None:
        return dz, None, dw_pre, None, None
    g = _rows(gate, M, rows_per_gate)
    p, dp, dw_post = y, alpha * g * dz, None
    dy = dp
    if post:
        n = y * r_post[:, None]
        w = 1.0 if w_post is None else w_post + off
        p, b = n * w, dp * w
        dy = r_post[:, None] * (b - n * (b * n).mean(1, keepdims=True))
        dw_post = (dp * n).sum(0)
    dgate = None
    if gate is not None:
        dgate = np.zeros_like(gate)
        np.add.at(dgate, np.arange(M) // rows_per_gate, alpha * dz * p)
    return dz, dy, dw_pre, dw_post, dgate


def rotary(x, turns, layout, scale=1.0, inverse=False):
    """x [M, H, hd], turns [M, rot / 2] (fractions of a full turn): the first rot elements of every
    head turned, as complex numbers."""
    rot = 2 * turns.shape[1]
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if layout == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    z = (a + 1j * b) * (scale * np.exp((-2j if inverse else 2j) * np.pi * turns))[:, None, :]
    y = x.copy()
    if layout == "half":
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    return y


def adamw(p, g, m, v, t, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01):
    """(p, m, v) after step t."""
    b1, b2 = betas
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    return p - lr * weight_decay * p - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps), m, v
