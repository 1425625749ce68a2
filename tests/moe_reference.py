"""Plain 64-bit restatements of the routed-layer operators, in numpy, one token or row at a
time where that is the clearest form.  Test infrastructure only."""
import math

import numpy as np

NEG = -np.inf


def bf16(a):
    """Round to bf16 (nearest even), as float64."""
    import torch

    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).bfloat16().double().numpy()


def route_scores(x, score):
    """Scores of one token's logits (float64), 0 where the logit is -inf."""
    x = np.asarray(x, dtype=np.float64)
    s = np.zeros_like(x)
    live = x > NEG
    if score == "sigmoid":
        s[live] = 1.0 / (1.0 + np.exp(-x[live]))
    elif live.any():
        m = x[live].max()
        e = np.where(x[live] == m, 1.0, np.exp(np.minimum(x[live] - m, 0.0)))
        s[live] = e / e.sum()
    return s


def route_token(x, K, bias=None, score="softmax", groups=1, top_groups=1, group_best=1,
                renorm=True, scale=1.0):
    """-> (experts list with -1 in empty slots, weights, least gap that settled the choice)."""
    x = np.asarray(x, dtype=np.float64)
    E = len(x)
    s = route_scores(x, score)
    v = x if bias is None else s + np.asarray(bias, dtype=np.float64)
    allowed = [e for e in range(E) if x[e] > NEG]
    gap = np.inf
    if groups > 1 and top_groups < groups:
        per = E // groups
        value = []
        for g in range(groups):
            mine = [e for e in allowed if e // per == g]
            if not mine:
                value.append(NEG)
                continue
            by = (lambda e: s[e]) if (group_best == 2 and bias is None) else (lambda e: v[e])
            best = sorted((by(e) for e in mine), reverse=True)[:group_best]
            value.append(float(sum(best)))
        order = sorted(range(groups), key=lambda g: (-value[g], g))
        kept = [g for g in order[:top_groups] if value[g] > NEG]
        if value[order[top_groups]] > NEG:
            gap = min(gap, value[order[top_groups - 1]] - value[order[top_groups]])
        allowed = [e for e in allowed if e // per in kept]
    order = sorted(allowed, key=lambda e: (-v[e], e))
    chosen = order[:K]
    for a, b in zip(order[:K], order[1:K + 1]):
        gap = min(gap, v[a] - v[b])
    w = np.zeros(K)
    if chosen:
        if renorm and score == "softmax":
            m = max(x[e] for e in chosen)
            p = np.array([1.0 if x[e] == m else math.exp(x[e] - m) for e in chosen])
            p /= p.sum()
        else:
            p = np.array([s[e] for e in chosen])
            if renorm:
                p = p / p.sum() if p.sum() > 0 else p * 0
        w[:len(chosen)] = scale * p
    return chosen + [-1] * (K - len(chosen)), w, gap


def route_weights(x, chosen, score, renorm, scale):
    """The weights of a fixed choice, differentiable in x (float64)."""
    s = route_scores(x, score)
    p = np.array([s[e] if e >= 0 else 0.0 for e in chosen])
    if renorm:
        p = p / p.sum() if p.sum() > 0 else p * 0
    return scale * p


def route_backward_token(x, chosen, dw, ds, score, renorm, scale):
    """dL/dx of one token by the chain rule through the full Jacobians."""
    x = np.asarray(x, dtype=np.float64)
    E = len(x)
    s = route_scores(x, score)
    if score == "softmax":
        J = np.diag(s) - np.outer(s, s)
    else:
        J = np.diag(s * (1.0 - s))
    G = np.zeros(E) if ds is None else np.where(x > NEG, np.asarray(ds, dtype=np.float64), 0.0)
    if dw is not None:
        live = [(k, e) for k, e in enumerate(chosen) if e >= 0 and x[e] > NEG]
        p = np.array([s[e] for _, e in live])
        g = scale * np.array([dw[k] for k, _ in live], dtype=np.float64)
        if renorm and p.sum() > 0:
            g = (g - (g * p).sum() / p.sum()) / p.sum()
        elif renorm:
            g = g * 0
        for (_, e), v in zip(live, g):
            G[e] += v
    dx = J @ G
    return np.where(x > NEG, dx, 0.0)


def dispatch(idx, E):
    idx = np.asarray(idx)
    T, K = idx.shape
    flat = idx.reshape(-1)
    rows = [[p for p in range(T * K) if flat[p] == e] for e in range(E)] if T * K < 3000 else None
    if rows is None:
        order = np.argsort(np.where(flat < 0, E, flat), kind="stable")
        counts = np.bincount(flat[flat >= 0], minlength=E)
        order = order[:counts.sum()]
    else:
        counts = np.array([len(r) for r in rows])
        order = np.array([p for r in rows for p in r], dtype=np.int64)
    off = np.concatenate([[0], np.cumsum(counts)])
    row_of = np.full(T * K, -1)
    row_of[order] = np.arange(len(order))
    row_index = np.full(T * K, -1)
    row_index[:len(order)] = order // K
    return off, row_index, row_of.reshape(T, K)


def _phi(x):
    return 0.5 * np.vectorize(math.erfc)(-np.asarray(x, dtype=np.float64) / math.sqrt(2.0)) \
        if np.size(x) else np.zeros_like(x, dtype=np.float64)


def _logistic(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def act(name, z):
    """Activation of pre-activations z [rows, N] in float64."""
    if name in ("swiglu", "geglu"):
        F = z.shape[1] // 2
        return act("silu" if name == "swiglu" else "gelu", z[:, :F]) * z[:, F:]
    return {"none": lambda: z, "relu": lambda: np.maximum(z, 0.0), "gelu": lambda: z * _phi(z),
            "silu": lambda: z * _logistic(z)}[name]()


def act_slope(name, z):
    if name == "relu":
        return (z > 0).astype(np.float64)
    if name == "gelu":
        return _phi(z) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "silu":
        s = _logistic(z)
        return s + z * s * (1.0 - s)
    return np.ones_like(z)


def act_backward(name, dy, z):
    if name in ("swiglu", "geglu"):
        inner = "silu" if name == "swiglu" else "gelu"
        F = z.shape[1] // 2
        gate, up = z[:, :F], z[:, F:]
        return np.concatenate([dy * up * act_slope(inner, gate), dy * act(inner, gate)], axis=1)
    return dy * act_slope(name, z)


def combine(y, row_of, w, residual):
    T, K = row_of.shape
    out = np.zeros((T, y.shape[1])) if residual is None else np.array(residual, dtype=np.float64)
    for k in range(K):
        has = row_of[:, k] >= 0
        wk = np.ones(T) if w is None else w[:, k].astype(np.float64)
        out[has] += wk[has, None] * y[row_of[has, k]]
    return out


def combine_backward(dout, y, row_of, w, M):
    T, K = row_of.shape
    dy = np.zeros((M, dout.shape[1]))
    dw = np.zeros((T, K))
    for k in range(K):
        has = np.nonzero(row_of[:, k] >= 0)[0]
        r = row_of[has, k]
        dy[r] = (1.0 if w is None else w[has, k:k + 1].astype(np.float64)) * dout[has]
        if y is not None:
            dw[has, k] = (dout[has] * y[r]).sum(axis=1)
    return dy, dw
