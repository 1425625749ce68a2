"""The adapter and gradient operators, case by case: inputs, the call, a plain form and a 64-bit one.

Three operators beside the grouped products:

* ``lora``      low-rank adapters of many requests (or of every expert) at once beside a shared
                projection: u[r] = x[t(r)] A[e]^T, out[o(r)] = base[o(r)] + scale[e] u[r] B[e]^T
                for the rows r of adapter e; rows of no adapter keep their base;
* ``lora_bwd``  its backward pass: v[r] = scale[e] dy[o(r)] B[e], dx[o(r)] = dx_base[o(r)] + v[r] A[e],
                dA[e] = sum of v[r]^T x[t(r)], dB[e] = scale[e] * sum of dy[o(r)]^T u[r];
* ``clip``      the norm of all gradients together, and the gradients scaled down to a largest norm.

``run`` computes one of them, with elementary torch operations when ``own`` is false and
through the library when it is true.  ``exact`` is the definition in 64 bits, written apart.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # A decode step of 16 requests, most with an adapter of their own out of 64 resident ones.
        {"name": "lora_decode", "op": "lora", "T": 16, "E": 64, "R": 16, "K": 4096, "N": 4096,
         "rows": "tokens", "none": 0.0, "skew": 0.0, "base": True, "save": False},
        # A larger decode batch, a wide projection, some requests without an adapter.
        {"name": "lora_decode_wide", "op": "lora", "T": 128, "E": 32, "R": 64, "K": 4096, "N": 8192,
         "rows": "tokens", "none": 0.1, "skew": 0.0, "base": True, "save": False},
        # Prompts of several requests (odd total) with popular and rare adapters.
        {"name": "lora_prefill", "op": "lora", "T": 4093, "E": 8, "R": 16, "K": 4096, "N": 1536,
         "rows": "tokens", "none": 0.1, "skew": 1.0, "base": True, "save": False},
        # Fine-tuning one adapter: all tokens of a training step.
        {"name": "lora_train", "op": "lora", "T": 16384, "E": 1, "R": 64, "K": 4096, "N": 4096,
         "rows": "plain", "none": 0.0, "skew": 0.0, "base": True, "save": True},
        # Fine-tuning an adapter per expert on the MoE FFN pair's up-projection: 8192 tokens,
        # eight of 64 experts each, x gathered, the rest in row order.
        {"name": "lora_experts", "op": "lora", "T": 8192, "E": 64, "R": 32, "K": 4096, "N": 1536,
         "rows": "routed", "none": 0.0, "skew": 0.5, "base": True, "save": True},
        # The backward pass: a small batch of odd length, the training step above, a skewed
        # batch of 16 adapters.
        {"name": "lora_bwd_small", "op": "lora_bwd", "T": 1021, "E": 4, "R": 8, "K": 2048, "N": 1536,
         "rows": "tokens", "none": 0.1, "skew": 0.0, "base": True},
        {"name": "lora_bwd_train", "op": "lora_bwd", "T": 16384, "E": 1, "R": 64, "K": 4096, "N": 4096,
         "rows": "plain", "none": 0.0, "skew": 0.0, "base": True},
        {"name": "lora_bwd_skew", "op": "lora_bwd", "T": 8192, "E": 16, "R": 16, "K": 4096, "N": 8192,
         "rows": "tokens", "none": 0.0, "skew": 1.0, "base": False},
        # The norm alone of one layer's router gradient: latency.
        {"name": "norm_router", "op": "clip", "count": 1, "lo": 64 * 4096, "hi": 64 * 4096,
         "dtype": "f32", "packed": False, "clip": False, "size": 1.0},
        # Clipping an adapter's gradients: two matrices of rank 16 for 64 projections.
        {"name": "clip_adapters", "op": "clip", "count": 128, "lo": 16 * 4096, "hi": 16 * 4096,
         "dtype": "bf16", "packed": False, "clip": True, "size": 1.0},
        # A model's gradients, bf16 and fp32 mixed, of odd sizes, packed one behind the other.
        {"name": "clip_mixed", "op": "clip", "count": 301, "lo": 1, "hi": 4000001,
         "dtype": "mixed", "packed": True, "clip": True, "size": 1e-3},
        # Expert weight gradients: 64 experts of 1536 x 4096.
        {"name": "clip_experts", "op": "clip", "count": 64, "lo": 1536 * 4096, "hi": 1536 * 4096,
         "dtype": "bf16", "packed": False, "clip": True, "size": 1.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["lora", "lora", "lora", "lora_bwd", "lora_bwd", "clip"])
    if op == "clip":
        lo = _log_int(rng, 1, 100000)
        hi = _log_int(rng, lo, 4000000)
        count = _log_int(rng, 1, min(1500, max(1, 200000000 // hi)))
        return {"op": "clip", "count": count, "lo": lo, "hi": hi,
                "dtype": rng.choice(["bf16", "f32", "mixed"]), "packed": rng.random() < 0.5,
                "clip": rng.random() < 0.7, "size": rng.choice([1.0, 1e-3, 1e-7])}
    K, N = 8 * _log_int(rng, 16, 1024), 8 * _log_int(rng, 16, 1024)
    rows = rng.choice(["tokens", "tokens", "plain", "routed"])
    # as much to read and write as the listed training step, at most
    most = (16384 * 8192) // (K + N) // (8 if rows == "routed" else 1)
    c = {"op": op, "T": _log_int(rng, 1, min(16384, most)), "E": _log_int(rng, 1, 128),
         "R": 8 * _log_int(rng, 1, 16), "K": K, "N": N, "rows": rows,
         "none": rng.choice([0.0, 0.1]) if rows != "routed" else 0.0,
         "skew": rng.choice([0.0, 1.0]), "base": rng.random() < 0.7}
    if op == "lora":
        c["save"] = rng.random() < 0.3
    return c


TOP_K = 8  # experts of a token where the rows are routed ones


# ---------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _row_tables(c, g):
    """adapter_off [E+1], the rows' tokens (None: row r is token r), counts, M.  Rows past
    adapter_off[E] have no adapter."""
    T, E = c["T"], c["E"]
    p = torch.arange(1, E + 1, device=DEV, dtype=torch.float32) ** -(1.5 * c["skew"])
    if c["rows"] == "routed":
        k = min(TOP_K, E)
        u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-12, 1 - 1e-7)
        which = torch.topk(torch.log(p) - torch.log(-torch.log(u)), k, dim=1).indices.flatten()
        token = torch.arange(T, device=DEV).repeat_interleave(k)
    else:
        which = torch.multinomial(p, T, replacement=True, generator=g)
        if c["none"] > 0:
            which = torch.where(torch.rand(T, generator=g, device=DEV) < c["none"], E, which)
        token = torch.arange(T, device=DEV)
    M = which.numel()
    counts = torch.bincount(which, minlength=E + 1).cpu().tolist()
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(counts[:E]), 0).int()
    order = torch.sort(which, stable=True).indices
    index = None if c["rows"] == "plain" else token[order].int()
    return off.to(DEV), index, counts, M


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] == "clip":
        _gradients(c, g, st)
        return st
    T, E, R, K, N = c["T"], c["E"], c["R"], c["K"], c["N"]
    st["off"], st["index"], st["counts"], M = _row_tables(c, g)
    st["M"] = M
    out_rows = M if c["rows"] == "routed" else T
    # where the rows of base, out, dy and dx lie: in row order, or at the tokens
    st["out_index"] = st["index"] if c["rows"] == "tokens" else None
    st["x"] = _randn(g, T, K).bfloat16()
    st["a"] = (_randn(g, E, R, K) * K ** -0.5).bfloat16()
    st["b"] = (_randn(g, E, N, R) * R ** -0.5).bfloat16()
    st["scale"] = torch.rand(E, generator=g, device=DEV) * 2 + 0.25
    if c["op"] == "lora":
        st["base"] = _randn(g, out_rows, N).bfloat16() if c["base"] else None
    else:
        st["dy"] = _randn(g, out_rows, N).bfloat16()
        st["dx_base"] = _randn(g, out_rows, K).bfloat16() if c["base"] else None
        # what the forward pass kept: u of every row with an adapter, zeros behind them
        u = torch.zeros(M, R, device=DEV)
        r = 0
        for e, n in enumerate(st["counts"][:E]):
            if n:
                u[r:r + n] = _take(st["x"], st["index"], r, n).float() @ st["a"][e].float().t()
            r += n
        st["u"] = u
    return st


def _sizes(c):
    """Sizes spread over lo .. hi, evenly in their logarithm, in an order that mixes them."""
    n = c["count"]
    if n == 1 or c["lo"] == c["hi"]:
        return [c["hi"]] * n
    f = math.log(c["hi"] / c["lo"]) / (n - 1)
    s = [max(c["lo"], min(c["hi"], int(c["lo"] * math.exp(f * i)))) for i in range(n)]
    return [s[(i * 7) % n] if n % 7 else s[i] for i in range(n)]


def _gradients(c, g, st):
    """Gradients as views of one buffer for each type, and the same views of an output buffer."""
    kinds = {"bf16": [torch.bfloat16], "f32": [torch.float32], "mixed": [torch.bfloat16, torch.float32]}
    kinds = kinds[c["dtype"]]
    at = {k: 0 for k in kinds}
    places = []
    for i, n in enumerate(_sizes(c)):
        k = kinds[i % len(kinds)]
        places.append((k, at[k], n))
        at[k] += n if c["packed"] else -(-n // 128) * 128
    st["flat"], st["out_flat"] = [], []
    views, outs = {}, {}
    for k in kinds:
        buf = torch.zeros(max(1, at[k]), dtype=k, device=DEV)
        for t0 in range(0, buf.numel(), 1 << 26):
            t1 = min(buf.numel(), t0 + (1 << 26))
            buf[t0:t1] = (_randn(g, t1 - t0) * c["size"]).to(k)
        st["flat"].append(buf)
        out = torch.zeros_like(buf)
        st["out_flat"].append(out)
        views[k], outs[k] = buf, out
    st["grads"] = [views[k][p:p + n] for k, p, n in places]
    st["outs"] = [outs[k][p:p + n] for k, p, n in places]
    for i in range(5, len(places), 17):  # parameters that a step did not reach
        st["grads"][i].zero_()
    st["max_norm"] = 0.5 * c["size"]
    if own:
        from moe_grouped_gemm_wgrad_gb300 import mgw
        # the tables of a model's gradient buffers, which a training loop keeps from step to step
        st["table"] = mgw.GradTable(st["grads"], out=st["outs"] if c["clip"] else None)


# ------------------------------------------------------------------------------ plain forms
def _take(t, index, r, n):
    return t[r:r + n] if index is None else t[index[r:r + n].long()]


def _plain_lora(st):
    c = st["case"]
    x, a, b, index, out_index = st["x"], st["a"], st["b"], st["index"], st["out_index"]
    M, N = st["M"], c["N"]
    out = torch.empty(M, N, dtype=torch.float32, device=x.device)
    u = torch.zeros(M, c["R"], dtype=torch.float32, device=x.device)
    r = 0
    for e, n in enumerate(st["counts"][:c["E"]]):
        if n:
            u[r:r + n] = _take(x, index, r, n).float() @ a[e].float().t()
            out[r:r + n] = (u[r:r + n] * st["scale"][e]) @ b[e].float().t()
        r += n
    out[r:] = 0
    if st["base"] is not None:
        out += _take(st["base"], out_index, 0, M).float()
    y = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
    if out_index is None:
        y.copy_(out)
    else:
        y[out_index.long()] = out.to(torch.bfloat16)
    return {"out": y, "u": u} if c["save"] else {"out": y}


def _plain_lora_bwd(st):
    c = st["case"]
    x, a, b, index, out_index = st["x"], st["a"], st["b"], st["index"], st["out_index"]
    M, K = st["M"], c["K"]
    dx = torch.empty(M, K, dtype=torch.float32, device=x.device)
    da = torch.zeros(a.shape, dtype=torch.bfloat16, device=x.device)
    db = torch.zeros(b.shape, dtype=torch.bfloat16, device=x.device)
    r = 0
    for e, n in enumerate(st["counts"][:c["E"]]):
        if n:
            dy = _take(st["dy"], out_index, r, n).float() * st["scale"][e]
            v = dy @ b[e].float()
            dx[r:r + n] = v @ a[e].float()
            da[e] = (v.t() @ _take(x, index, r, n).float()).to(torch.bfloat16)
            db[e] = (dy.t() @ st["u"][r:r + n]).to(torch.bfloat16)
        r += n
    dx[r:] = 0
    if st["dx_base"] is not None:
        dx += _take(st["dx_base"], out_index, 0, M).float()
    y = torch.empty(M, K, dtype=torch.bfloat16, device=x.device)
    if out_index is None:
        y.copy_(dx)
    else:
        y[out_index.long()] = dx.to(torch.bfloat16)
    return {"dx": y, "da": da, "db": db}


def _plain_clip(st):
    c = st["case"]
    sums = [(t.float() * t.float()).sum() for t in st["grads"]]
    norm = torch.sqrt(torch.stack(sums).double().sum()).float().reshape(1)
    if not c["clip"]:
        return {"norm": norm}
    coef = torch.clamp(st["max_norm"] / (norm + EPS), max=1.0)
    for t, o in zip(st["grads"], st["outs"]):
        o.copy_(t.float() * coef)
    return {"norm": norm, "out": st["out_flat"]}


# ------------------------------------------------------------------------------------ calls
def run(state):
    c = state["case"]
    if not own:
        return {"lora": _plain_lora, "lora_bwd": _plain_lora_bwd, "clip": _plain_clip}[c["op"]](state)
    from moe_grouped_gemm_wgrad_gb300 import mgw
    st = state
    if c["op"] == "lora":
        out = mgw.grouped_lora(st["x"], st["a"], st["b"], st["off"], row_index=st["index"],
                               out_index=st["out_index"], scale=st["scale"], base=st["base"],
                               save_u=c["save"])
        return {"out": out[0], "u": out[1]} if c["save"] else {"out": out}
    if c["op"] == "lora_bwd":
        dx, da, db = mgw.grouped_lora_backward(st["dy"], st["x"], st["u"], st["a"], st["b"], st["off"],
                                               row_index=st["index"], out_index=st["out_index"],
                                               scale=st["scale"], dx_base=st["dx_base"])
        return {"dx": dx, "da": da, "db": db}
    if not c["clip"]:
        return {"norm": mgw.grad_norm(st["table"])}
    norm = mgw.clip_grads(st["table"], st["max_norm"])
    return {"norm": norm, "out": st["out_flat"]}


# ----------------------------------------------------------------------------------- bounds
def work(case):
    c = case
    if c["op"] == "clip":
        bytes_ = {"bf16": [2], "f32": [4], "mixed": [2, 4]}[c["dtype"]]
        sizes = _sizes(c)
        b = sum(n * bytes_[i % len(bytes_)] for i, n in enumerate(sizes))
        n = sum(sizes)
        return {"bytes": 2 * b if c["clip"] else b, "flops": 3 * n if c["clip"] else 2 * n}
    T, E, R, K, N = c["T"], c["E"], c["R"], c["K"], c["N"]
    M = T * min(TOP_K, E) if c["rows"] == "routed" else T
    used = E * (1 - (1 - 1 / E) ** M) if E > 1 else 1
    weights = used * R * (K + N) * 2
    tables = 4 * (E + 1) + (0 if c["rows"] == "plain" else 4 * M)
    if c["op"] == "lora":
        b = T * K * 2 + M * N * 2 * (2 if c["base"] else 1) + weights + tables
        b += 4 * M * R if c["save"] else 0
        return {"bytes": int(b), "flops": 2 * M * R * (K + N)}
    b = T * K * 2 + M * N * 2 + M * K * 2 * (2 if c["base"] else 1) + weights + tables + 4 * M * R
    return {"bytes": int(b + E * R * (K + N) * 2), "flops": 4 * M * R * (K + N)}


# ---------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    c = case
    if c["op"] == "clip":
        total = torch.zeros((), dtype=torch.float64, device=DEV)
        for t in st["grads"]:
            for s in t.split(1 << 26):
                total += torch.linalg.vector_norm(s.double()) ** 2
        norm = total.sqrt()
        if not c["clip"]:
            return {"norm": norm.reshape(1)}
        f = min(1.0, st["max_norm"] / (float(norm) + EPS))
        outs = []
        for buf, o in zip(st["flat"], st["out_flat"]):
            y = torch.zeros(buf.shape, dtype=torch.float64, device=DEV)
            outs.append((buf, y))
        for t in st["grads"]:
            for buf, y in outs:
                if t.dtype == buf.dtype:
                    p = t.storage_offset()
                    y[p:p + t.numel()] = t.double() * f
        return {"norm": norm.reshape(1), "out": [y for _, y in outs]}
    E, M, off = c["E"], st["M"], st["off"].tolist()
    rows = torch.arange(M, device=DEV)
    tok = rows if st["index"] is None else st["index"].long()
    dst = rows if st["out_index"] is None else st["out_index"].long()

    def each():
        for e in range(E):
            for r0 in range(off[e], off[e + 1], 8192):
                r1 = min(off[e + 1], r0 + 8192)
                yield e, tok[r0:r1], dst[r0:r1], slice(r0, r1)

    if c["op"] == "lora":
        y = torch.zeros(M, c["N"], dtype=torch.float64, device=DEV)
        if st["base"] is not None:
            y[dst] = st["base"].double()[dst]
        u = torch.zeros(M, c["R"], dtype=torch.float64, device=DEV)
        for e, t, d, r in each():
            u[r] = torch.einsum("tk,rk->tr", st["x"][t].double(), st["a"][e].double())
            y[d] += torch.einsum("tr,nr->tn", u[r], st["b"][e].double()) * st["scale"][e].double()
        return {"out": y, "u": u} if c["save"] else {"out": y}
    dx = torch.zeros(M, c["K"], dtype=torch.float64, device=DEV)
    if st["dx_base"] is not None:
        dx[dst] = st["dx_base"].double()[dst]
    da = torch.zeros(st["a"].shape, dtype=torch.float64, device=DEV)
    db = torch.zeros(st["b"].shape, dtype=torch.float64, device=DEV)
    for e, t, d, r in each():
        s, g = st["scale"][e].double(), st["dy"][d].double()
        v = torch.einsum("tn,nr->tr", g, st["b"][e].double()) * s
        dx[d] += torch.einsum("tr,rk->tk", v, st["a"][e].double())
        da[e] += torch.einsum("tr,tk->rk", v, st["x"][t].double())
        db[e] += torch.einsum("tn,tr->nr", g, st["u"][r].double()) * s
    return {"dx": dx, "da": da, "db": db}
