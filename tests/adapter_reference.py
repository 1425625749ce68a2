"""The adapter operators and the gradient norm, restated in 64 bits row by row and value by value,
without the library; test_adapter_reference.py checks these against difference quotients."""
import numpy as np


def lora(x, a, b, off, t, o, scale, base):
    """-> (out, u) for rows r of adapter e: t[r] the row of x, o[r] that of base and out (-1: none)."""
    out = np.zeros((base.shape[0], b.shape[1])) if base.ndim == 1 else base.copy()
    u = np.zeros((len(t), a.shape[1]))
    for e in range(len(off) - 1):
        for r in range(off[e], off[e + 1]):
            u[r] = a[e] @ x[t[r]] if t[r] >= 0 else 0
            if o[r] >= 0:
                out[o[r]] = out[o[r]] + scale[e] * (b[e] @ u[r])
    return out, u


def lora_backward(dy, x, u, a, b, off, t, o, scale, dx_base):
    dx, da, db = dx_base.copy(), np.zeros_like(a), np.zeros_like(b)
    for e in range(len(off) - 1):
        for r in range(off[e], off[e + 1]):
            g = dy[o[r]] if o[r] >= 0 else np.zeros(b.shape[1])
            v = g @ b[e]
            if o[r] >= 0:
                dx[o[r]] = dx[o[r]] + scale[e] * (v @ a[e])
            if t[r] >= 0:
                da[e] += scale[e] * np.outer(v, x[t[r]])
            db[e] += scale[e] * np.outer(g, u[r])
    return dx, da, db


def norm(tensors):
    return float(np.sqrt(sum(float(np.sum(t.astype(np.longdouble) ** 2)) for t in tensors)))
