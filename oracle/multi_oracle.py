"""Plain fp64 reference of a projection whose rows have different adapters, and of the norms and clipping
of grouped gradients.  Like lora_oracle it shares no code with the CUDA path."""
import numpy as np


def multi_fwd(X, W0, A, B, s, ids, bias=None):
    """(Y, Z): y_i = x_i W0^T + s_a z_i B_a^T (+ bias), z_i = x_i A_a^T, a = ids[i]; none outside 0 .. n - 1."""
    Y, Z = X @ W0.T, np.zeros((X.shape[0], A.shape[1]))
    for i, a in enumerate(ids):
        if 0 <= a < len(A):
            Z[i] = A[a] @ X[i]
            Y[i] += s[a] * (B[a] @ Z[i])
    return Y if bias is None else Y + bias, Z


def multi_bwd(X, W0, A, B, s, ids, Z, dY):
    """(dX, dA, dB, dbias, G) from Z as the forward left it; G the gradients of the z_i."""
    dX, dA, dB = dY @ W0, np.zeros_like(A), np.zeros_like(B)
    G = np.zeros((X.shape[0], A.shape[1]))
    for i, a in enumerate(ids):
        if 0 <= a < len(A):
            G[i] = s[a] * (dY[i] @ B[a])
            dX[i] += G[i] @ A[a]
            dA[a] += np.outer(G[i], X[i])
            dB[a] += s[a] * np.outer(dY[i], Z[i])
    return dX, dA, dB, dY.sum(0), G


def clip(grads, max_norm, groups, count):
    """(norms, clipped): norms[g] over the tensors of group g, each scaled by min(1, max_norm / (norm + 1e-6)),
    or zero where the group's norm is not finite.  max_norm None: left as they are."""
    sq = np.zeros(count)
    for g, k in zip(grads, groups):
        sq[k] += (g ** 2).sum()
    norms = np.sqrt(sq)
    out = []
    for g, k in zip(grads, groups):
        if max_norm is None:
            out.append(g)
        elif np.isfinite(norms[k]):
            out.append(g * min(1.0, max_norm / (norms[k] + 1e-6)))
        else:
            out.append(np.zeros_like(g))
    return norms, out
