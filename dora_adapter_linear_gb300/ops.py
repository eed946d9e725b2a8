"""Convenience layer over the C ABI: allocates outputs and workspaces with PyTorch, then calls
the entry point of the same name.  PyTorch is used only for device memory and the stream."""
from __future__ import annotations

import math
import threading
from ctypes import c_float
from functools import lru_cache

import torch

from . import _lib as L
from .adapters import AdapterPlan, adapter_plan  # noqa: F401
from .rotary import rotary_plan  # noqa: F401

_WS = {}


def workspace(nbytes: int, device) -> torch.Tensor:
    """A cached scratch buffer of at least nbytes, its error word cleared when it is made.  It belongs to
      this thread and stream: a call's launches run without the interpreter's lock, so those of two threads'
        calls on one stream come in any order, and each has to find the partial results of its own call;
      this graph capture, if the stream is in one: the graph keeps the address, in memory from its own pool,
        whatever is called later, and no other graph or call writes there."""
    if not isinstance(device, torch.device):
        device = torch.device("cuda", device) if isinstance(device, int) else torch.device(device)
    L.need_current("the operands", device)
    stream = L.current_stream(device)
    capture, thread = L.capture_id(stream), threading.get_ident()
    key = (device, stream, thread, capture)
    buf = _WS.get(key)
    if buf is None or buf.numel() < nbytes:
        for k in [k for k in list(_WS) if k[2] == thread and k[3] not in (0, capture)]:
            del _WS[k]          # of captures that have ended: their graphs' pools keep the memory
        new = torch.empty if capture else torch.zeros       # in a graph: the error word's 256 bytes alone
        old, buf = buf, new(max(nbytes, 256), dtype=torch.uint8, device=device)
        if capture:
            buf[:256].zero_()
        elif old is not None:
            buf[:256].copy_(old[:256])          # an error that has not been looked at yet
        _WS[key] = buf
    return buf


def check_device_errors():
    """Waits for the device, then raises LoraError if a wait inside a kernel ran out since the last check: calls
    launch and return, so this is where it shows, and the outputs of the calls before are not to be used.
    Looks at the calls of every thread and stream, of captured ones at those of the last capture."""
    torch.cuda.synchronize()
    failed = 0
    for buf in list(_WS.values()):
        status = L.lora_check_device_error(buf)
        if status:
            failed = status
            L.lora_clear_device_error(buf)
    if failed:
        raise L.LoraError(failed, "a call since the last check")


def _shape_of(X, W0, A):
    return L.shape(X.shape[0], X.shape[1], W0.shape[0], A.shape[0], L.dtype_code(X))


def _check_linear(X, W0, A, B, bias=None, Z=None, dY=None, Y=None):
    """The kernels trust the shapes they are given (tensor maps and strides come from them), so a
    mismatched tensor would be read out of bounds: check every operand against X [M, in],
    W0 [out, in], A [r, in] before anything is launched."""
    if X.dim() != 2 or W0.dim() != 2:
        raise ValueError("X and W0 must be 2-D")
    M, d_in = X.shape
    d_out, r = W0.shape[0], A.shape[0]
    want = {"W0": (W0, (d_out, d_in)), "A": (A, (r, d_in)), "B": (B, (d_out, r)), "bias": (bias, (d_out,)),
            "Z": (Z, (M, r)), "dY": (dY, (M, d_out)), "Y": (Y, (M, d_out))}
    if W0.shape[1] != d_in:
        raise ValueError(f"W0 {tuple(W0.shape)} does not match X {tuple(X.shape)}")
    for name, (t, shape) in [("X", (X, (M, d_in)))] + list(want.items()):
        if t is None:
            continue
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
        if t.dtype != X.dtype or t.device != X.device or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {X.dtype} tensor on {X.device}")


def _check_like(name, t, shape, X):
    """t (if given) must have `shape`, X's dtype and device, and a contiguous layout."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != X.dtype or t.device != X.device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {X.dtype} tensor on {X.device}")


def _check_mlp(X, g, u, d, saved=None, dY=None):
    """Each projection has its own rank: A [r, n_in], B [n_out, r] with r = A.shape[0]."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, H = X.shape
    I = g["W"].shape[0]
    for nm, p, n_out, n_in in (("gate", g, I, H), ("up", u, I, H), ("down", d, H, I)):
        r = p["A"].shape[0]
        _check_like(nm + " W", p["W"], (n_out, n_in), X)
        _check_like(nm + " A", p["A"], (r, n_in), X)
        _check_like(nm + " B", p["B"], (n_out, r), X)
    rg, ru, rd = g["A"].shape[0], u["A"].shape[0], d["A"].shape[0]
    if saved is not None:
        for k in ("e", "u", "h"):
            _check_like(k, saved[k], (M, I), X)
        _check_like("Zgu", saved["Zgu"], (M, rg + ru), X)
        _check_like("Zd", saved["Zd"], (M, rd), X)
    _check_like("dY", dY, (M, H), X)


def _mlp_shape(X, g, u, d, act):
    M, H = X.shape
    return L.mlp_shape(M, H, g["W"].shape[0], g["A"].shape[0], u["A"].shape[0], d["A"].shape[0], act=act)


def _check_qkv(X, W0, leaves, bias=None, Z=None, dY=None):
    if X.dim() != 2 or W0.dim() != 2 or not leaves:
        raise ValueError("X and W0 must be 2-D and there must be at least one leaf")
    M, d_in = X.shape
    r = leaves[0][0].shape[0]
    N = sum(B.shape[0] for _, B, _ in leaves)
    _check_like("W0", W0, (N, d_in), X)
    for l, (A, B, _) in enumerate(leaves):
        _check_like(f"A{l}", A, (r, d_in), X)
        _check_like(f"B{l}", B, (B.shape[0], r), X)
    _check_like("bias", bias, (N,), X)
    _check_like("Z", Z, (M, len(leaves) * r), X)
    _check_like("dY", dY, (M, N), X)


def _check_shapes(ref, **named):
    """Each named tensor (None allowed) must have the given shape and dtype, ref's device and a
    contiguous layout; named values are (tensor, shape, dtype) triples.  The kernels read every
    operand with the element size its dtype implies, so a wrong dtype is an out-of-bounds read."""
    for name, (t, shape, dtype) in named.items():
        if t is None:
            continue
        if (tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != ref.device
                or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on {ref.device}, "
                             f"got {tuple(t.shape)} {t.dtype} on {t.device}")


def _check_vec(name, t, n, X, dtype):
    """t (if given) must be a contiguous [n] tensor of `dtype` on X's device."""
    if t is not None and (tuple(t.shape) != (n,) or t.dtype != dtype or t.device != X.device
                          or not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous [{n}] {dtype} tensor on {X.device}, "
                         f"got {tuple(t.shape)} {t.dtype} on {t.device}")


F32 = torch.float32
BF16 = torch.bfloat16


def lora_linear_fwd(X, W0, A, B, s, bias=None, save_z=True):
    _check_linear(X, W0, A, B, bias)
    sh = _shape_of(X, W0, A)
    Y = torch.empty(X.shape[0], W0.shape[0], dtype=X.dtype, device=X.device)
    Z = torch.empty(X.shape[0], A.shape[0], dtype=X.dtype, device=X.device) if save_z else None
    ws = workspace(L.lora_workspace_bytes(L.OP_LINEAR_FWD, sh), X.device)
    L.lora_linear_fwd(sh, X, W0, A, B, bias, s, Y, Z, ws)
    return Y, Z


def lora_linear_bwd(X, W0, A, B, Z, dY, s, need_dx=True, need_dbias=False):
    _check_linear(X, W0, A, B, Z=Z, dY=dY)
    sh = _shape_of(X, W0, A)
    dX = torch.empty_like(X) if need_dx else None
    dA = torch.empty_like(A)
    dB = torch.empty_like(B)
    dbias = torch.empty(W0.shape[0], dtype=X.dtype, device=X.device) if need_dbias else None
    ws = workspace(L.lora_workspace_bytes(L.OP_LINEAR_BWD, sh), X.device)
    L.lora_linear_bwd(sh, X, W0, A, B, Z, dY, s, dX, dA, dB, dbias, ws)
    return dX, dA, dB, dbias


def _check_mask(mask, X):
    if (mask.dtype != torch.uint8 or tuple(mask.shape) != tuple(X.shape) or not mask.is_contiguous()
            or mask.device != X.device):
        raise ValueError(f"dropout mask must be contiguous uint8 {tuple(X.shape)}, got {mask.dtype} "
                         f"{tuple(mask.shape)}")


def lora_linear_dropout_fwd(X, mask, keep_scale, W0, A, B, s, bias=None, save_z=True):
    """mask: uint8 [M, d_in] (1 = kept), keep_scale = 1 / (1 - p)."""
    _check_linear(X, W0, A, B, bias)
    _check_mask(mask, X)
    sh = _shape_of(X, W0, A)
    Y = torch.empty(X.shape[0], W0.shape[0], dtype=X.dtype, device=X.device)
    Z = torch.empty(X.shape[0], A.shape[0], dtype=X.dtype, device=X.device) if save_z else None
    ws = workspace(L.lora_workspace_bytes(L.OP_DROPOUT_FWD, sh), X.device)
    L.lora_linear_dropout_fwd(sh, X, mask, keep_scale, W0, A, B, bias, s, Y, Z, ws)
    return Y, Z


def lora_linear_dropout_bwd(X, mask, keep_scale, W0, A, B, Z, dY, s, need_dx=True, need_dbias=False):
    _check_linear(X, W0, A, B, Z=Z, dY=dY)
    _check_mask(mask, X)
    sh = _shape_of(X, W0, A)
    dX = torch.empty_like(X) if need_dx else None
    dA = torch.empty_like(A)
    dB = torch.empty_like(B)
    dbias = torch.empty(W0.shape[0], dtype=X.dtype, device=X.device) if need_dbias else None
    ws = workspace(L.lora_workspace_bytes(L.OP_DROPOUT_BWD, sh), X.device)
    L.lora_linear_dropout_bwd(sh, X, mask, keep_scale, W0, A, B, Z, dY, s, dX, dA, dB, dbias, ws)
    return dX, dA, dB, dbias


def dora_rownorm2(W0):
    _need_cuda("W0", W0)
    sh = L.shape(0, W0.shape[1], W0.shape[0], 8, L.dtype_code(W0))
    r0 = torch.empty(W0.shape[0], dtype=torch.float32, device=W0.device)
    L.dora_rownorm2(sh, W0, r0)
    return r0


def dora_linear_fwd(X, W0, A, B, m, r0, s, eps=1e-12, bias=None, save_z=True):
    _check_linear(X, W0, A, B, bias)
    _check_vec("m", m, W0.shape[0], X, X.dtype)
    _check_vec("r0", r0, W0.shape[0], X, F32)
    sh = _shape_of(X, W0, A)
    dev = X.device
    Y = torch.empty(X.shape[0], W0.shape[0], dtype=X.dtype, device=dev)
    Z = torch.empty(X.shape[0], A.shape[0], dtype=X.dtype, device=dev) if save_z else None
    n = torch.empty(W0.shape[0], dtype=torch.float32, device=dev)
    V = torch.empty(W0.shape[0], A.shape[0], dtype=torch.float32, device=dev)
    ws = workspace(L.lora_workspace_bytes(L.OP_DORA_FWD, sh), dev)
    L.dora_linear_fwd(sh, X, W0, A, B, m, bias, r0, s, eps, Y, Z, n, V, ws)
    return Y, Z, n, V


def dora_linear_bwd(X, W0, A, B, m, bias, Y, Z, n, V, dY, s, eps=1e-12, need_dx=True, need_dbias=False):
    _check_linear(X, W0, A, B, bias, Z=Z, dY=dY, Y=Y)
    _check_vec("m", m, W0.shape[0], X, X.dtype)
    _check_vec("n", n, W0.shape[0], X, F32)
    _check_shapes(X, V=(V, (W0.shape[0], A.shape[0]), F32))
    sh = _shape_of(X, W0, A)
    dX = torch.empty_like(X) if need_dx else None
    dA = torch.empty_like(A)
    dB = torch.empty_like(B)
    dm = torch.empty_like(m)
    dbias = torch.empty(W0.shape[0], dtype=X.dtype, device=X.device) if need_dbias else None
    ws = workspace(L.lora_workspace_bytes(L.OP_DORA_BWD, sh), X.device)
    L.dora_linear_bwd(sh, X, W0, A, B, m, bias, Y, Z, n, V, dY, s, eps, dX, dA, dB, dm, dbias, ws)
    return dX, dA, dB, dm, dbias


def dora_colnorm2(W0):
    _need_cuda("W0", W0)
    sh = L.shape(0, W0.shape[1], W0.shape[0], 8, L.dtype_code(W0))
    c0 = torch.empty(W0.shape[1], dtype=torch.float32, device=W0.device)
    L.dora_colnorm2(sh, W0, c0)
    return c0


def dora_cols_fwd(X, W0, A, B, m, c0, s, eps=1e-12, bias=None, save_z=True):
    """m, c0: [d_in].  Returns Y, Z, n [d_in], U [d_in, r] (the last three saved for the backward)."""
    _check_linear(X, W0, A, B, bias)
    _check_vec("m", m, W0.shape[1], X, X.dtype)
    _check_vec("c0", c0, W0.shape[1], X, F32)
    sh = _shape_of(X, W0, A)
    dev = X.device
    Y = torch.empty(X.shape[0], W0.shape[0], dtype=X.dtype, device=dev)
    Z = torch.empty(X.shape[0], A.shape[0], dtype=X.dtype, device=dev) if save_z else None
    n = torch.empty(W0.shape[1], dtype=torch.float32, device=dev)
    U = torch.empty(W0.shape[1], A.shape[0], dtype=torch.float32, device=dev)
    ws = workspace(L.lora_workspace_bytes(L.OP_DORA_COLS_FWD, sh), dev)
    L.dora_cols_fwd(sh, X, W0, A, B, m, bias, c0, s, eps, Y, Z, n, U, ws)
    return Y, Z, n, U


def dora_cols_bwd(X, W0, A, B, m, Z, n, U, dY, s, eps=1e-12, need_dx=True, need_dbias=False):
    _check_linear(X, W0, A, B, Z=Z, dY=dY)
    _check_vec("m", m, W0.shape[1], X, X.dtype)
    _check_vec("n", n, W0.shape[1], X, F32)
    _check_shapes(X, U=(U, (W0.shape[1], A.shape[0]), F32))
    sh = _shape_of(X, W0, A)
    dX = torch.empty_like(X) if need_dx else None
    dA = torch.empty_like(A)
    dB = torch.empty_like(B)
    dm = torch.empty_like(m)
    dbias = torch.empty(W0.shape[0], dtype=X.dtype, device=X.device) if need_dbias else None
    ws = workspace(L.lora_workspace_bytes(L.OP_DORA_COLS_BWD, sh), X.device)
    L.dora_cols_bwd(sh, X, W0, A, B, m, Z, n, U, dY, s, eps, dX, dA, dB, dm, dbias, ws)
    return dX, dA, dB, dm, dbias


def lora_mlp_swiglu_fwd(X, g, u, d, act=0):
    """g, u, d: dicts with W, A, B, s; act 0 SwiGLU, 1 GeGLU.  Returns (Y, saved) where saved
    holds e, u, h, Zgu, Zd."""
    _check_mlp(X, g, u, d)
    M, H = X.shape
    I = g["W"].shape[0]
    sh = _mlp_shape(X, g, u, d, act)
    dev = X.device
    e_ = torch.empty(M, I, dtype=X.dtype, device=dev)
    u_ = torch.empty_like(e_)
    h_ = torch.empty_like(e_)
    Zgu = torch.empty(M, sh.r_g + sh.r_u, dtype=X.dtype, device=dev)
    Zd = torch.empty(M, sh.r_d, dtype=X.dtype, device=dev)
    Y = torch.empty(M, H, dtype=X.dtype, device=dev)
    ws = workspace(L.lora_mlp_workspace_bytes(L.OP_MLP_FWD, sh), dev)
    pg, pu, pd = (L.proj(p["W"], p["A"], p["B"], p["s"]) for p in (g, u, d))
    L.lora_mlp_swiglu_fwd(sh, X, pg, pu, pd, Y, e_, u_, h_, Zgu, Zd, ws)
    return Y, {"e": e_, "u": u_, "h": h_, "Zgu": Zgu, "Zd": Zd}


def lora_mlp_swiglu_bwd(X, g, u, d, saved, dY, need_dx=True, act=0):
    _check_mlp(X, g, u, d, saved, dY)
    sh = _mlp_shape(X, g, u, d, act)
    dX = torch.empty_like(X) if need_dx else None
    grads = {k: torch.empty_like(v) for k, v in
             (("dAg", g["A"]), ("dBg", g["B"]), ("dAu", u["A"]), ("dBu", u["B"]), ("dAd", d["A"]), ("dBd", d["B"]))}
    ws = workspace(L.lora_mlp_workspace_bytes(L.OP_MLP_BWD, sh), X.device)
    pg, pu, pd = (L.proj(p["W"], p["A"], p["B"], p["s"]) for p in (g, u, d))
    L.lora_mlp_swiglu_bwd(sh, X, pg, pu, pd, saved["e"], saved["u"], saved["h"], saved["Zgu"], saved["Zd"], dY, dX,
                          grads["dAg"], grads["dBg"], grads["dAu"], grads["dBu"], grads["dAd"], grads["dBd"], ws)
    grads["dX"] = dX
    return grads


def w8a8_quantize_rows(X, A=None):
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    rows, cols = X.shape
    _check_shapes(X, X=(X, (rows, cols), BF16), A=(A, (None if A is None else A.shape[0], cols), BF16))
    _need_cuda("X", X)
    Xq = torch.empty(rows, cols, dtype=torch.int8, device=X.device)
    sx = torch.empty(rows, dtype=torch.float32, device=X.device)
    Z = torch.empty(rows, A.shape[0], dtype=X.dtype, device=X.device) if A is not None else None
    L.w8a8_quantize_rows(rows, cols, X, Xq, sx, A, 0 if A is None else A.shape[0], Z)
    return Xq, sx, Z


def w8a8_lora_bwd(X, Wq, sw, A, B, Z, dY, s, need_dx=True, need_dbias=False):
    M, d_in = X.shape
    d_out, r = Wq.shape[0], A.shape[0]
    if Wq.dtype != torch.int8:
        raise ValueError("Wq must be int8")
    _check_shapes(X, X=(X, (M, d_in), BF16), Wq=(Wq, (d_out, d_in), torch.int8), sw=(sw, (d_out,), F32),
                  A=(A, (r, d_in), BF16), B=(B, (d_out, r), BF16), Z=(Z, (M, r), BF16), dY=(dY, (M, d_out), BF16))
    dX = torch.empty_like(X) if need_dx else None
    dA = torch.empty_like(A)
    dB = torch.empty_like(B)
    dbias = torch.empty(d_out, dtype=X.dtype, device=X.device) if need_dbias else None
    ws = workspace(L.w8a8_bwd_workspace_bytes(M, d_in, d_out, r), X.device)
    L.w8a8_lora_bwd(M, d_in, d_out, r, X, Wq, sw, A, B, Z, dY, s, dX, dA, dB, dbias, ws)
    return dX, dA, dB, dbias


def w8a8_lora_fwd(Xq, sx, Wq, sw, Z, B, s, bias=None, want_acc=False, want_y=True):
    M, d_in = Xq.shape
    d_out = Wq.shape[0]
    r = 0 if Z is None else Z.shape[1]
    if Xq.dtype != torch.int8 or Wq.dtype != torch.int8:
        raise ValueError("Xq and Wq must be int8")
    _check_shapes(Xq, Xq=(Xq, (M, d_in), torch.int8), sx=(sx, (M,), F32), Wq=(Wq, (d_out, d_in), torch.int8),
                  sw=(sw, (d_out,), F32), Z=(Z, (M, r), BF16), B=(B, (d_out, r), BF16), bias=(bias, (d_out,), BF16))
    Y = torch.empty(M, d_out, dtype=torch.bfloat16, device=Xq.device) if want_y else None
    acc = torch.empty(M, d_out, dtype=torch.int32, device=Xq.device) if want_acc else None
    ws = workspace(L.w8a8_workspace_bytes(M, d_in, d_out), Xq.device)
    L.w8a8_lora_fwd(M, d_in, d_out, r, Xq, sx, Wq, sw, Z, B, s, bias, Y, acc, ws)
    return Y, acc


def lora_qkv_fwd(X, W0, leaves, bias=None, save_z=True):
    """leaves: [(A_l, B_l, s_l)] for the leaves of the fused weight W0 (rows in leaf order)."""
    _check_qkv(X, W0, leaves, bias)
    M, d_in = X.shape
    n = [B.shape[0] for _, B, _ in leaves]
    r = leaves[0][0].shape[0]
    sh = L.qkv_shape(M, d_in, n, r)
    Y = torch.empty(M, sum(n), dtype=X.dtype, device=X.device)
    Z = torch.empty(M, len(leaves) * r, dtype=X.dtype, device=X.device) if save_z else None
    ws = workspace(L.lora_qkv_workspace_bytes(L.OP_QKV_FWD, sh), X.device)
    L.lora_qkv_fwd(sh, X, W0, L.adapters(leaves), bias, Y, Z, ws)
    return Y, Z


def lora_qkv_bwd(X, W0, leaves, Z, dY, need_dx=True, need_dbias=False):
    _check_qkv(X, W0, leaves, Z=Z, dY=dY)
    M, d_in = X.shape
    n = [B.shape[0] for _, B, _ in leaves]
    r = leaves[0][0].shape[0]
    sh = L.qkv_shape(M, d_in, n, r)
    dX = torch.empty_like(X) if need_dx else None
    dA = [torch.empty_like(A) for A, _, _ in leaves]
    dB = [torch.empty_like(B) for _, B, _ in leaves]
    dbias = torch.empty(sum(n), dtype=X.dtype, device=X.device) if need_dbias else None
    ws = workspace(L.lora_qkv_workspace_bytes(L.OP_QKV_BWD, sh), X.device)
    L.lora_qkv_bwd(sh, X, W0, L.adapters(leaves), Z, dY, dX, dA, dB, dbias, ws)
    return dX, dA, dB, dbias


def w8a8_quantize_rows_bf16(X, A=None):
    """Per-token quantisation with the codes returned as bf16 values: (Xcodes, sx, Z)."""
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    rows, cols = X.shape
    _check_shapes(X, X=(X, (rows, cols), BF16), A=(A, (None if A is None else A.shape[0], cols), BF16))
    _need_cuda("X", X)
    Xc = torch.empty(rows, cols, dtype=torch.bfloat16, device=X.device)
    sx = torch.empty(rows, dtype=torch.float32, device=X.device)
    Z = torch.empty(rows, A.shape[0], dtype=X.dtype, device=X.device) if A is not None else None
    L.w8a8_quantize_rows_bf16(rows, cols, X, Xc, sx, A, 0 if A is None else A.shape[0], Z)
    return Xc, sx, Z


def w8a8_prepack_weight(Wq, sw, codes=True, dequant=True):
    """The frozen int8 weight laid out once: Wb the codes as bf16 for the forward, Wd the
    dequantised weight for the backward (each None when not asked for)."""
    if Wq.dtype != torch.int8 or Wq.dim() != 2:
        raise ValueError("Wq must be a 2-D int8 tensor")
    d_out, d_in = Wq.shape
    _check_shapes(Wq, Wq=(Wq, (d_out, d_in), torch.int8), sw=(sw, (d_out,), F32))
    _need_cuda("Wq", Wq)
    mk = lambda: torch.empty(d_out, d_in, dtype=torch.bfloat16, device=Wq.device)  # noqa: E731
    Wb = mk() if codes else None
    Wd = mk() if dequant else None
    L.w8a8_prepack_weight(d_out, d_in, Wq, sw, Wb, Wd)
    return Wb, Wd


def w8a8_lora_fwd_packed(Xc, sx, Wb, sw, Z, B, s, bias=None, want_acc=False, want_y=True):
    """w8a8_lora_fwd on prepacked operands (Xc from w8a8_quantize_rows_bf16, Wb from
    w8a8_prepack_weight)."""
    M, d_in = Xc.shape
    d_out = Wb.shape[0]
    r = 0 if Z is None else Z.shape[1]
    _check_shapes(Xc, Xc=(Xc, (M, d_in), BF16), sx=(sx, (M,), F32), Wb=(Wb, (d_out, d_in), BF16),
                  sw=(sw, (d_out,), F32), Z=(Z, (M, r), BF16), B=(B, (d_out, r), BF16), bias=(bias, (d_out,), BF16))
    Y = torch.empty(M, d_out, dtype=torch.bfloat16, device=Xc.device) if want_y else None
    acc = torch.empty(M, d_out, dtype=torch.int32, device=Xc.device) if want_acc else None
    ws = workspace(L.w8a8_packed_workspace_bytes(M, d_out), Xc.device)
    L.w8a8_lora_fwd_packed(M, d_in, d_out, r, Xc, sx, Wb, sw, Z, B, s, bias, Y, acc, ws)
    return Y, acc


def _row_stride(name, t, X):
    """The row stride of t: a tensor of X's shape [M, D], dtype and device with rows of consecutive
    elements, any stride of at least D between them."""
    if t.shape != X.shape or t.dtype is not X.dtype or t.device != X.device:
        raise ValueError(f"{name} must be a {tuple(X.shape)} {X.dtype} tensor on {X.device}, got {tuple(t.shape)} "
                         f"{t.dtype} on {t.device}")
    M, D = t.shape
    if t.is_contiguous() or M <= 1 and (D <= 1 or t.stride(1) == 1):
        return D
    ld, step = t.stride()
    if (step != 1 and D > 1) or ld < D:
        raise ValueError(f"{name} must have rows of consecutive elements that do not overlap, got strides {t.stride()}")
    return ld


def _rows_like(X):
    """A new contiguous tensor like X [M, D]."""
    return torch.empty_like(X) if X.is_contiguous() else torch.empty(X.shape, dtype=X.dtype, device=X.device)


def _need_cuda(name, t):
    """t must be where the call runs."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor, got one on {t.device}")
    L.need_current(name, t.device)


def _gate_rows(gate, rows_per_gate, X):
    """Rows that share a gate row; by default the rows of X split evenly over the gate's."""
    M, D = X.shape
    if gate.dim() != 2 or (gate.shape[0] == 0 and M > 0):
        raise ValueError("gate must be [rows, D]")
    G = gate.shape[0]
    if rows_per_gate is None:
        if G and M % G:
            raise ValueError(f"{M} rows do not split evenly over {G} gate rows: give rows_per_gate")
        rows_per_gate = max(M // max(G, 1), 1)
    if rows_per_gate < 1 or G != -(-M // rows_per_gate):
        raise ValueError(f"gate must have a row for every {rows_per_gate} of {M} rows, got {G}")
    _check_like("gate", gate, (G, D), X)
    return rows_per_gate


def _norm_shape(X, w_pre, w_post, gate, rows_per_gate, alpha, eps, w_offset, post_norm):
    if X.dim() != 2:
        raise ValueError("X must be 2-D")
    M, D = X.shape
    for name, w in (("w_pre", w_pre), ("w_post", w_post)):
        if w is not None and (w.shape != (D,) or w.dtype is not X.dtype or w.device != X.device
                              or not w.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous [{D}] {X.dtype} tensor on {X.device}, got {tuple(w.shape)} "
                             f"{w.dtype} on {w.device}")
    if w_post is not None and not post_norm:
        raise ValueError("w_post needs post_norm=True")
    per = 0 if gate is None else _gate_rows(gate, rows_per_gate, X)
    return L.LoraNormShape(M, D, per, D, D, D, D, alpha, eps, w_offset, 1 if post_norm else 0, L.dtype_code(X))


def _done(result, where):
    """The outputs of a call that the host module has made, or its error."""
    if type(result) is int:
        raise L.LoraError(result, where)
    return result


@lru_cache(maxsize=256)
def _norm_bwd_bytes(M, D, dtype, device):
    """Bytes of workspace; they go by the multiprocessors of the current device, of index `device`."""
    if dtype not in (BF16, F32):
        return 0
    return L.block_norm_bwd_workspace_bytes(L.LoraNormShape(M, D, 1, D, D, D, D, 1.0, 1.0, 0.0, 0,
                                                            L.LORA_BF16 if dtype == BF16 else L.LORA_F32))


def block_norm_fwd(X, Y=None, w_pre=None, w_post=None, gate=None, rows_per_gate=None, alpha=1.0, eps=1e-6,
                   w_offset=0.0, pre_norm=True, post_norm=False):
    """The end of one block and the start of the next: Xout = X + alpha gate o p with p the block
    output Y, normed (RMS, weight w_post) first when post_norm, and H = the RMS norm of Xout (weight
    w_pre) when pre_norm.  Weights are used as w + w_offset.  gate [G, D]: row i takes gate row
    i // rows_per_gate (by default the rows split evenly over the gate's).  Returns
    (Xout, H, r_pre, r_post); Xout is X when there is no Y, and what is not formed is None."""
    done = L.host().block_norm_fwd(X, Y, w_pre, w_post, gate, rows_per_gate, alpha, eps, w_offset, pre_norm, post_norm)
    if done is not None:
        return _done(done, "block_norm_fwd")
    sh = _norm_shape(X, w_pre, w_post, gate, rows_per_gate, alpha, eps, w_offset, post_norm)
    if Y is None and (gate is not None or post_norm or not pre_norm):
        raise ValueError("without a block output Y only the pre norm can be asked for")
    if w_pre is not None and not pre_norm:
        raise ValueError("w_pre needs pre_norm=True")
    sh.ldx = _row_stride("X", X, X)
    if Y is not None:
        sh.ldy = _row_stride("Y", Y, X)
    _need_cuda("X", X)
    M, dev = sh.M, X.device
    Xout = None if Y is None else _rows_like(X)
    H = _rows_like(X) if pre_norm else None
    r_pre = torch.empty(M, dtype=F32, device=dev) if pre_norm else None
    r_post = torch.empty(M, dtype=F32, device=dev) if post_norm else None
    L.block_norm_fwd(sh, X, Y, w_pre, w_post, gate, Xout, H, r_pre, r_post)
    return X if Y is None else Xout, H, r_pre, r_post


def block_norm_bwd(Xout, Y, r_pre, r_post, dH, dXout, w_pre=None, w_post=None, gate=None, rows_per_gate=None,
                   alpha=1.0, w_offset=0.0, post_norm=False, need_dx=True, need_dw=True, need_dgate=True):
    """Gradients of block_norm_fwd from those of H (dH) and Xout (dXout; either may be None): returns
    (dX, dY, dw_pre, dw_post, dgate), None for what is not asked for or has no input.  eps is in r_pre
    and r_post."""
    if Xout.dim() == 2 and Xout.is_cuda:
        need = _norm_bwd_bytes(*Xout.shape, Xout.dtype, L.current_device())
        if need:
            done = L.host().block_norm_bwd(Xout, Y, r_pre, r_post, dH, dXout, w_pre, w_post, gate, rows_per_gate, alpha,
                                           w_offset, post_norm, need_dx, need_dw, need_dgate,
                                           workspace(need, Xout.device))
            if done is not None:
                return _done(done, "block_norm_bwd")
    sh = _norm_shape(Xout, w_pre, w_post, gate, rows_per_gate, alpha, 1.0, w_offset, post_norm)
    M = sh.M
    if dH is None and dXout is None:
        raise ValueError("at least one of dH and dXout is needed")
    if Y is None and (gate is not None or post_norm):
        raise ValueError("a gate or post norm needs the block output Y")
    _check_vec("r_pre", r_pre, M, Xout, F32)
    _check_vec("r_post", r_post, M, Xout, F32)
    if (dH is not None and r_pre is None) or (post_norm and r_post is None):
        raise ValueError("r_pre (with dH) and r_post (with post_norm) come from the forward")
    sh.ldx = _row_stride("Xout", Xout, Xout)
    if Y is not None:
        sh.ldy = _row_stride("Y", Y, Xout)
    if dH is not None:
        sh.lddh = _row_stride("dH", dH, Xout)
    if dXout is not None:
        sh.lddz = _row_stride("dXout", dXout, Xout)
    _need_cuda("Xout", Xout)
    dev = Xout.device
    dX = _rows_like(Xout) if need_dx else None
    dY = _rows_like(Xout) if Y is not None else None
    dw_pre = torch.empty_like(w_pre) if need_dw and w_pre is not None else None
    dw_post = torch.empty_like(w_post) if need_dw and w_post is not None else None
    dgate = torch.empty_like(gate) if need_dgate and gate is not None else None
    ws = workspace(L.block_norm_bwd_workspace_bytes(sh), dev)
    L.block_norm_bwd(sh, Xout, Y, w_pre, w_post, gate, r_pre, r_post, dH, dXout, dX, dY, dw_pre, dw_post, dgate, ws)
    return dX, dY, dw_pre, dw_post, dgate


def _rotary(inverse, X, pos, plan, out):
    done = L.host().rotary(inverse, X, pos, plan.freq, plan.rot_dim, plan.scale, plan.layout, out)
    if done is not None:
        return _done(done, "rotary_bwd" if inverse else "rotary_fwd")
    if X.dim() != 3:
        raise ValueError(f"the heads must be [tokens, heads, head_dim], got {tuple(X.shape)}")
    M, H, hd = X.shape
    xt, xh, step = X.stride()
    if step != 1 and hd > 1:
        raise ValueError(f"a head must be consecutive elements, got strides {X.stride()}")
    wide = pos.dtype is torch.int64
    if pos.dim() != 1 or pos.shape[0] != M or not (wide or pos.dtype is torch.int32) or not pos.is_contiguous():
        raise ValueError(f"pos must be a contiguous [{M}] int32 or int64 tensor, got {tuple(pos.shape)} {pos.dtype}")
    dev = X.device
    if pos.device != dev or plan.freq.device != dev:
        raise ValueError(f"pos and the plan must be on {dev}")
    _check_shapes(X, **{"the plan's freq": (plan.freq, (plan.rot_dim // 2,), torch.int64)})
    if out is not None and out.requires_grad and torch.is_grad_enabled():
        raise ValueError("out needs a gradient, which would not be that of this call: call it under torch.no_grad()")
    if plan.rot_dim > hd:
        raise ValueError(f"the plan turns {plan.rot_dim} elements of a head, the heads have {hd}")
    _need_cuda("X", X)
    given = out
    if out is None:
        out = torch.empty(M, H, hd, dtype=X.dtype, device=dev)
    elif out is not X and (out.shape != X.shape or out.dtype is not X.dtype or out.device != dev
                           or (out.stride(2) != 1 and hd > 1)):
        raise ValueError(f"out must be like the heads, {tuple(X.shape)} {X.dtype} on {dev}")
    yt, yh = (xt, xh) if out is X else (out.stride(0), out.stride(1))
    sh = L.LoraRotaryShape(M, H, hd, plan.rot_dim, xt, xh, yt, yh, plan.scale, plan.layout, 64 if wide else 32,
                           L.dtype_code(X))
    (L.rotary_bwd if inverse else L.rotary_fwd)(sh, X, pos, plan.freq, out)
    if given is not None and not out.is_inference():
        torch.autograd.graph.increment_version(out)     # autograd notices if it had kept it for a backward
    return out


def rotary_fwd(X, pos, plan, out=None):
    """Turns the heads X [tokens, heads, head_dim] (any token and head stride: the query and key heads
    of a packed projection are one view) by their positions pos [tokens]; `plan` from rotary_plan.
    out=X turns in place; by default a new contiguous tensor is returned.  Any other out may not have an
    element of X among its own."""
    return _rotary(False, X, pos, plan, out)


def rotary_bwd(dY, pos, plan, out=None):
    """The gradient of rotary_fwd: the turn by the negative angle, with the same scale."""
    return _rotary(True, dY, pos, plan, out)


def _multi_shape(X, W0, A, B, s, plan, bias=None, Z=None, dY=None):
    """The shape of a call with a stack of adapters, its operands checked against X [M, in], W0 [out, in] and
    A [n, r, in]."""
    if X.dim() != 2 or W0.dim() != 2 or A.dim() != 3:
        raise ValueError("X and W0 must be 2-D and A a stack of adapters [n, r, in]")
    if not isinstance(plan, AdapterPlan):
        raise ValueError("plan must come from adapter_plan()")
    M, d_in = X.shape
    d_out, (n, r, _) = W0.shape[0], A.shape
    for name, t, shape in (("X", X, (M, d_in)), ("W0", W0, (d_out, d_in)), ("A", A, (n, r, d_in)),
                           ("B", B, (n, d_out, r)), ("bias", bias, (d_out,)), ("Z", Z, (M, r)), ("dY", dY, (M, d_out))):
        _check_like(name, t, shape, X)
    if isinstance(s, torch.Tensor):
        _check_vec("s", s, n, X, F32)
    elif not math.isfinite(c_float(s).value):           # as the kernels have it
        raise ValueError(f"s must be finite, got {s}")
    if plan.rows != M or plan.adapters != n:
        raise ValueError(f"the plan is of {plan.rows} rows and {plan.adapters} adapters, the call has {M} and {n}")
    if plan.buffer.device != X.device:
        raise ValueError(f"the plan must be on {X.device}, it is on {plan.buffer.device}")
    return L.LoraMultiShape(M, d_in, d_out, r, n, L.dtype_code(X))


def _need_filled(plan):
    if not plan.filled:
        raise ValueError("the plan holds no ids yet: make it by adapter_plan() or call update()")


@lru_cache(maxsize=1024)
def _multi_bytes(backward, M, d_in, d_out, r, n, dtype):
    """Bytes of workspace; 0 for what the calls do not take."""
    if dtype not in (BF16, F32):
        return 0
    sh = L.LoraMultiShape(M, d_in, d_out, r, n, L.LORA_BF16 if dtype == BF16 else L.LORA_F32)
    return L.lora_multi_workspace_bytes(backward, sh)


def _multi_workspace(backward, X, W0, A, plan):
    """The workspace of a call whose operands look well, or None: what is wrong is for the checks to name."""
    if X.dim() == 2 and W0.dim() == 2 and A.dim() == 3 and X.is_cuda and isinstance(plan, AdapterPlan) \
            and plan.filled:
        need = _multi_bytes(backward, *X.shape, W0.shape[0], A.shape[1], A.shape[0], X.dtype)
        if need:
            return workspace(need, X.device)
    return None


def lora_multi_fwd(X, W0, A, B, s, plan, bias=None, save_z=True):
    """The projection of a batch whose rows have different adapters: row i takes adapter ids[i] of the stacks
    A [n, r, in] and B [n, out, r], or the frozen base alone where it has none; `plan` from
    adapter_plan(ids, n).  s: a number, or an fp32 tensor [n] with one for each adapter.  Returns (Y, Z)."""
    ws = _multi_workspace(False, X, W0, A, plan)
    if ws is not None:
        done = L.host().multi_fwd(X, W0, A, B, s, plan.buffer, plan.rows, plan.adapters, bias, save_z, ws)
        if done is not None:
            return _done(done, "lora_multi_fwd")
    sh = _multi_shape(X, W0, A, B, s, plan, bias)
    _need_cuda("X", X)
    _need_filled(plan)
    Y = torch.empty(sh.M, sh.d_out, dtype=X.dtype, device=X.device)
    Z = torch.empty(sh.M, sh.r, dtype=X.dtype, device=X.device) if save_z else None
    ws = workspace(L.lora_multi_workspace_bytes(False, sh), X.device)
    L.lora_multi_fwd(sh, X, W0, A, B, bias, s, plan.buffer, Y, Z, ws)
    return Y, Z


def lora_multi_bwd(X, W0, A, B, Z, dY, s, plan, need_dx=True, need_dbias=False):
    """Gradients of lora_multi_fwd with W0 frozen: (dX, dA, dB, dbias), dA and dB stacks like A and B, zeros
    for an adapter without rows.  Z: from the forward, or None to recompute it (bf16 with up to 256 rows: an
    element may then be the forward's neighbour, its fp32 sum being formed in another order)."""
    ws = _multi_workspace(True, X, W0, A, plan)
    if ws is not None:
        done = L.host().multi_bwd(X, W0, A, B, Z, dY, s, plan.buffer, plan.rows, plan.adapters, need_dx, need_dbias, ws)
        if done is not None:
            return _done(done, "lora_multi_bwd")
    sh = _multi_shape(X, W0, A, B, s, plan, Z=Z, dY=dY)
    _need_cuda("X", X)
    _need_filled(plan)
    dX = torch.empty_like(X) if need_dx else None
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    dbias = torch.empty(sh.d_out, dtype=X.dtype, device=X.device) if need_dbias else None
    ws = workspace(L.lora_multi_workspace_bytes(True, sh), X.device)
    L.lora_multi_bwd(sh, X, W0, A, B, Z, dY, s, plan.buffer, dX, dA, dB, dbias, ws)
    return dX, dA, dB, dbias
