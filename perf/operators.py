"""The routed-layer operators, case by case: inputs, the call, a plain form and a 64-bit one.

Five operators of a Mixture-of-Experts layer surround the grouped GEMMs:

* ``route``     logits [T, E] -> the K experts of every token and their weights, and the
                gradient of the weights (and of the scores) back to the logits;
* ``dispatch``  the experts of every token -> expert_off, row_index (the row order the
                quantizers gather by) and row_of (where each (token, slot) pair went);
* ``ffn``       the grouped MXFP8 product with bias, activation (gated ones too) and residual
                in its epilogue;
* ``act``       its backward pass up to the products: dz = dy * act'(z), and the bias gradient
                summed over every expert's rows;
* ``combine``   out[t] = residual[t] + sum_k w[t, k] y[row_of[t, k]], and its backward pass.

``run`` computes one of them, with elementary torch operations when ``own`` is false and
through the library when it is true.  ``exact`` is the definition in 64 bits, written apart.
"""
import math

import torch

own = False

DEV = "cuda"
NEG = float("-inf")
GATED = ("swiglu", "geglu")


def listed():
    return [
        # A decode step of a few sequences: the router's latency.
        {"name": "route_decode", "op": "route", "T": 4, "E": 64, "K": 8, "dtype": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renorm": True,
         "scale": 1.0, "train": False, "masked": 0.0},
        # A long prompt (odd length) through a group-limited sigmoid router with balance bias.
        {"name": "route_prefill_groups", "op": "route", "T": 8191, "E": 256, "K": 8,
         "dtype": "f32", "score": "sigmoid", "bias": True, "groups": 8, "top_groups": 4,
         "renorm": True, "scale": 2.5, "train": False, "masked": 0.0},
        # A training step's tokens, softmax without renormalisation, an auxiliary loss on the
        # scores: forward and backward.
        {"name": "route_train", "op": "route", "T": 65536, "E": 64, "K": 8, "dtype": "bf16",
         "score": "softmax", "bias": False, "groups": 1, "top_groups": 1, "renorm": False,
         "scale": 1.0, "train": True, "masked": 0.0},
        # The row tables of a decode step and of a large training batch with skewed experts.
        {"name": "dispatch_decode", "op": "dispatch", "T": 16, "K": 8, "E": 64, "skew": 0.0,
         "dropped": 0.0},
        {"name": "dispatch_train", "op": "dispatch", "T": 131072, "K": 8, "E": 64, "skew": 1.0,
         "dropped": 0.0},
        # One decode step: 16 tokens, eight of 64 experts each, all weights read for few rows.
        {"name": "ffn_decode", "op": "ffn", "M": 128, "E": 64, "N": 2048, "Kd": 4096,
         "act": "swiglu", "bias": False, "residual": False, "save": False, "skew": 0.0},
        # The MoE FFN pair's up-projection (8192 tokens, top-8 of 64 experts, 1536 x 4096), as a
        # training step runs it: bias, GELU, the pre-activation kept.
        {"name": "ffn_train_pair", "op": "ffn", "M": 65536, "E": 64, "N": 1536, "Kd": 4096,
         "act": "gelu", "bias": True, "residual": False, "save": True, "skew": 0.0},
        # The same layer's backward pass at the activation, with the bias gradient; and a
        # ragged gated one.
        {"name": "act_train_pair", "op": "act", "M": 65536, "E": 64, "N": 1536, "act": "gelu",
         "bias": True, "skew": 0.0},
        {"name": "act_gated_ragged", "op": "act", "M": 5003, "E": 16, "N": 4096, "act": "swiglu",
         "bias": True, "skew": 1.0},
        # Back to token order: a decode step with its residual, an odd fp32 one, and a training
        # step of the MoE FFN pair in both directions.
        {"name": "combine_decode", "op": "combine", "T": 16, "K": 8, "H": 4096, "dtype": "bf16",
         "residual": True, "train": False, "dropped": 0.0},
        {"name": "combine_odd_f32", "op": "combine", "T": 1021, "K": 4, "H": 1999, "dtype": "f32",
         "residual": True, "train": False, "dropped": 0.05},
        {"name": "combine_train_pair", "op": "combine", "T": 8192, "K": 8, "H": 4096,
         "dtype": "bf16", "residual": True, "train": True, "dropped": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["route", "route", "dispatch", "ffn", "ffn", "act", "combine", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log_int(rng, max(2, 8 // groups), 512 // groups)
        T = _log_int(rng, 1, min(65536, (65536 * 64) // E))
        top_groups = rng.randint(1, groups)
        K = rng.randint(1, min(16, E // groups * top_groups))
        return {"op": "route", "T": T, "E": E, "K": K, "dtype": rng.choice(["bf16", "f32"]),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5,
                "groups": groups, "top_groups": top_groups, "renorm": rng.random() < 0.6,
                "scale": rng.choice([1.0, 2.5]), "train": rng.random() < 0.5,
                "masked": rng.choice([0.0, 0.0, 0.2])}
    if op == "dispatch":
        return {"op": "dispatch", "T": _log_int(rng, 1, 131072), "K": rng.randint(1, 8),
                "E": _log_int(rng, 1, 512), "skew": rng.choice([0.0, 1.0]),
                "dropped": rng.choice([0.0, 0.0, 0.1])}
    if op == "ffn":
        N, Kd = 256 * _log_int(rng, 1, 16), 128 * _log_int(rng, 1, 32)
        E = _log_int(rng, 1, min(64, (64 * 1536 * 4096) // (N * Kd)))
        M = _log_int(rng, 1, min(65536, (65536 * 1536 * 4096) // (2 * N * Kd)))
        return {"op": "ffn", "M": M, "E": E, "N": N, "Kd": Kd,
                "act": rng.choice(["none", "relu", "gelu", "silu", "swiglu", "geglu"]),
                "bias": rng.random() < 0.5, "residual": rng.random() < 0.3,
                "save": rng.random() < 0.5, "skew": rng.choice([0.0, 1.0])}
    if op == "act":
        N = 256 * _log_int(rng, 1, 16)
        return {"op": "act", "M": _log_int(rng, 1, min(65536, 65536 * 1536 // N)),
                "E": _log_int(rng, 1, 64), "N": N,
                "act": rng.choice(["relu", "gelu", "silu", "swiglu", "geglu"]),
                "bias": rng.random() < 0.7, "skew": rng.choice([0.0, 1.0])}
    dtype = rng.choice(["bf16", "bf16", "f32"])
    H, K = _log_int(rng, 64, 4096), rng.randint(1, 8)
    cap = (8192 * 8 * 4096) // (K * H) // (2 if dtype == "f32" else 1)
    return {"op": "combine", "T": _log_int(rng, 1, min(8192, cap)), "K": K, "H": H,
            "dtype": dtype, "residual": rng.random() < 0.5, "train": rng.random() < 0.5,
            "dropped": rng.choice([0.0, 0.05])}


# ---------------------------------------------------------------------------------- inputs
def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _pick_experts(g, T, K, E, skew):
    """Distinct experts per token; with skew, expert e is drawn about (e+1)^-skew as often."""
    pop = -skew * torch.log(torch.arange(1, E + 1, device=DEV, dtype=torch.float32))
    out = torch.empty(T, K, dtype=torch.int32, device=DEV)
    for t0 in range(0, T, 16384):
        t1 = min(T, t0 + 16384)
        u = torch.rand(t1 - t0, E, generator=g, device=DEV).clamp_(1e-12, 1 - 1e-7)
        out[t0:t1] = torch.topk(pop - torch.log(-torch.log(u)), K, dim=1).indices.int()
    return out


def _split(g, M, E, skew):
    """Rows per expert: M rows thrown at E experts, unevenly when skew is set."""
    p = torch.arange(1, E + 1, device=DEV, dtype=torch.float32) ** -(1.5 * skew)
    e = torch.multinomial(p, M, replacement=True, generator=g)
    counts = torch.bincount(e, minlength=E).cpu().tolist()
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(counts), 0).int()
    return counts, off.to(DEV)


def _drop(g, idx, share):
    if share > 0:
        idx[torch.rand(idx.shape, generator=g, device=DEV) < share] = -1
    return idx


def _route_gap(c, logits, bias):
    """Per token, how far the choice is from being settled by rounding (float64): the least
    distance between neighbouring selection values among the chosen and the first not chosen,
    and between the last group kept and the first left out."""
    T, E, K = c["T"], c["E"], c["K"]
    x = logits.double()
    if c["score"] == "softmax":
        s = torch.softmax(x, 1)
    else:
        s = torch.sigmoid(x)
    sel = (s + bias.double()).masked_fill(x == NEG, NEG)
    gap = torch.full((x.shape[0],), 1.0, dtype=torch.float64, device=DEV)
    if c["groups"] > 1:
        per = sel.view(-1, c["groups"], E // c["groups"])
        best = torch.topk(per, min(2, per.shape[2]), dim=2).values
        gs = torch.where(best == NEG, 0.0, best).sum(2).masked_fill(best[:, :, 0] == NEG, NEG)
        srt = torch.sort(gs, 1, descending=True).values
        if c["top_groups"] < c["groups"]:
            d = srt[:, c["top_groups"] - 1] - srt[:, c["top_groups"]]
            gap = torch.minimum(gap, torch.nan_to_num(d, nan=1.0))
        keep = gs >= srt[:, c["top_groups"] - 1:c["top_groups"]]
        sel = sel.masked_fill(~keep.repeat_interleave(E // c["groups"], 1), NEG)
    v = torch.topk(sel, min(E, K + 1), dim=1).values
    if v.shape[1] > 1:
        d = torch.nan_to_num(v[:, :-1] - v[:, 1:], nan=1.0, posinf=1.0)
        gap = torch.minimum(gap, d.min(1).values)
    return gap


def _route_inputs(c, g):
    T, E = c["T"], c["E"]
    bias = None
    if c["bias"]:
        # a balance bias moves by a fixed step per update
        bias = torch.round(_randn(g, E) * 40) * 1e-3

    def fresh(n):
        x = (_randn(g, n, E) * 1.5).to(_dtype(c["dtype"]))
        if c["masked"] > 0:  # experts that a token may not use; now and then all of them
            x = x.masked_fill(torch.rand(n, E, generator=g, device=DEV) < c["masked"], NEG)
            x[torch.rand(n, generator=g, device=DEV) < 0.02] = NEG
        return x

    logits = fresh(T)
    if bias is not None:
        # Where two sums score + bias lie within a rounding of each other, the rounding and not
        # the operator settles which comes first: such tokens are drawn again.
        for _ in range(40):
            bad = (_route_gap(c, logits, bias) < 2e-6).nonzero().flatten()
            if bad.numel() == 0:
                break
            logits[bad] = fresh(bad.numel())
    return logits, bias


def _quantize(rows):
    """Row-wise MXFP8 of fp32 rows [R, C]: e4m3 bytes and one e8m0 byte per 32 columns."""
    R, C = rows.shape
    b = rows.view(R, C // 32, 32)
    amax = b.abs().amax(2)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 9, torch.full_like(amax, -127).int())
    e = e.clamp(-127, 127)
    q = torch.ldexp(b, -e.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).reshape(R, C), (e + 127).to(torch.uint8)


def _atoms(sc):
    """Scale bytes [R, C/32] (R a multiple of 128) in 512-byte atoms: by 128-column chunk, then
    128-row tile; inside, row r0 + 32 r1 and block kb at 16 r0 + 4 r1 + kb."""
    R, B = sc.shape
    return sc.view(R // 128, 4, 32, B // 4, 4).permute(3, 0, 2, 1, 4).contiguous().flatten()


def _from_atoms(flat, R, C):
    return flat[:R * C // 32].view(C // 128, R // 128, 32, 4, 4).permute(1, 3, 2, 0, 4) \
        .reshape(R, C // 32)


def _capacity(M, E):
    return (M + 127 * E + 127) // 128 * 128


def _ffn_inputs(c, g):
    M, E, N, Kd = c["M"], c["E"], c["N"], c["Kd"]
    counts, off = _split(g, M, E, c["skew"])
    mcap = _capacity(M, E)
    xq = torch.zeros(mcap, Kd, dtype=torch.uint8, device=DEV)
    xsc = torch.zeros(mcap, Kd // 32, dtype=torch.uint8, device=DEV)
    p = 0
    for n in counts:
        if n:
            xq[p:p + n], xsc[p:p + n] = _quantize(_randn(g, n, Kd).bfloat16().float())
        p += (n + 127) // 128 * 128
    mw = _capacity(E * N, E)
    wq = torch.zeros(mw, Kd, dtype=torch.uint8, device=DEV)
    wsc = torch.zeros(mw, Kd // 32, dtype=torch.uint8, device=DEV)
    for e in range(E):
        w = (_randn(g, N, Kd) * Kd ** -0.5).bfloat16().float()
        wq[e * N:(e + 1) * N], wsc[e * N:(e + 1) * N] = _quantize(w)
    out_f = N // 2 if c["act"] in GATED else N
    return {"xq": xq, "xs": _atoms(xsc), "wq": wq, "ws": _atoms(wsc), "off": off,
            "counts": counts,
            "bias": _randn(g, E, N) * 0.5 if c["bias"] else None,
            "residual": _randn(g, M, out_f).bfloat16() if c["residual"] else None}


def prepare(case, seed):
    c, g = case, _gen(seed)
    st = {"case": c}
    if c["op"] == "route":
        st["logits"], st["bias"] = _route_inputs(c, g)
        if c["train"]:
            st["dweights"] = _randn(g, c["T"], c["K"])
            # a balance loss is a mean over the tokens: every token's share is small
            st["dscores"] = _randn(g, c["T"], c["E"]) * 1e-2
    elif c["op"] == "dispatch":
        K = min(c["K"], c["E"])
        st["idx"] = _drop(g, _pick_experts(g, c["T"], K, c["E"], c["skew"]), c["dropped"])
    elif c["op"] == "ffn":
        st.update(_ffn_inputs(c, g))
    elif c["op"] == "act":
        out_f = c["N"] // 2 if c["act"] in GATED else c["N"]
        st["counts"], st["off"] = _split(g, c["M"], c["E"], c["skew"])
        st["z"] = _randn(g, c["M"], c["N"]).bfloat16()
        st["dy"] = _randn(g, c["M"], out_f).bfloat16()
    else:
        T, K, H = c["T"], c["K"], c["H"]
        dt = _dtype(c["dtype"])
        # the rows of 64 experts' segments: a stable order by expert
        e = _drop(g, torch.randint(0, 64, (T, K), generator=g, device=DEV), c["dropped"]).flatten()
        order = torch.sort(torch.where(e < 0, 64, e), stable=True).indices
        rows = torch.empty_like(order)
        rows[order] = torch.arange(T * K, device=DEV)
        st["row_of"] = torch.where(e < 0, -1, rows).int().view(T, K)
        M = int((e >= 0).sum())
        st["y"] = _randn(g, M, H).to(dt)
        w = torch.rand(T, K, generator=g, device=DEV) + 0.05
        st["weights"] = w / w.sum(1, keepdim=True)
        st["residual"] = _randn(g, T, H).to(dt) if c["residual"] else None
        if c["train"]:
            st["dout"] = _randn(g, T, H).to(dt)
    return st


# ------------------------------------------------------------------------------ plain forms
def _plain_route(st):
    c = st["case"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    x = st["logits"].float()
    masked = x == NEG
    if c["score"] == "softmax":
        top = x.max(1, keepdim=True).values
        ex = torch.exp(x - torch.where(top == NEG, 0.0, top))
        tot = ex.sum(1, keepdim=True)
        s = ex / torch.where(tot == 0, 1.0, tot)
    else:
        s = 1.0 / (1.0 + torch.exp(-x))
    # both scores grow with the logit, so without a bias the logits give the order
    sel = x if st["bias"] is None else (s + st["bias"]).masked_fill(masked, NEG)
    if G > 1:
        per = sel.view(T, G, E // G)
        first = per.max(2)
        gs = first.values
        if st["bias"] is not None and E // G > 1:
            rest = per.scatter(2, first.indices.unsqueeze(2), NEG).max(2).values
            gs = gs + torch.where(rest == NEG, 0.0, rest)
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        for _ in range(c["top_groups"]):
            j = gs.argmax(1, keepdim=True)
            keep.scatter_(1, j, True)
            gs = gs.scatter(1, j, NEG)
        sel = sel.masked_fill(~keep.repeat_interleave(E // G, 1), NEG)
    else:
        sel = sel.clone()
    idx = torch.empty(T, K, dtype=torch.int64, device=x.device)
    none = torch.empty(T, K, dtype=torch.bool, device=x.device)
    for k in range(K):
        m = sel.max(1, keepdim=True)
        idx[:, k:k + 1] = m.indices
        none[:, k:k + 1] = m.values == NEG
        sel.scatter_(1, m.indices, NEG)
    xs = x.gather(1, idx).masked_fill(none, NEG)
    ss = s.gather(1, idx).masked_fill(none, 0.0)
    if c["renorm"]:
        if c["score"] == "softmax":
            top = xs.max(1, keepdim=True).values
            ss = torch.exp(xs - torch.where(top == NEG, 0.0, top))
        tot = ss.sum(1, keepdim=True)
        ss = ss / torch.where(tot == 0, 1.0, tot)
    w = ss * c["scale"]
    out = {"expert_idx": idx.masked_fill(none, -1).int(), "weights": w}
    if not c["train"]:
        return out
    out["scores"] = s.masked_fill(masked, 0.0)
    dw = st["dweights"] * c["scale"]
    s_sel = s.gather(1, idx).masked_fill(none, 0.0)
    if c["renorm"]:
        ws = w / c["scale"]
        inner = dw - (dw * ws).sum(1, keepdim=True)
    # gradient at the scores' inputs: first through the auxiliary loss, then the weights
    d = st["dscores"].masked_fill(masked, 0.0)
    sm = out["scores"]
    if c["score"] == "softmax":
        dx = sm * (d - (sm * d).sum(1, keepdim=True))
        if c["renorm"]:
            dx = dx.scatter_add(1, idx, (ws * inner).masked_fill(none, 0.0))
        else:
            dx = dx - sm * (dw * s_sel).sum(1, keepdim=True)
            dx = dx.scatter_add(1, idx, (dw * s_sel).masked_fill(none, 0.0))
    else:
        dx = d * sm * (1.0 - sm)
        # 1 - s and, renormalised, s / sum = ws
        if c["renorm"]:
            dx = dx.scatter_add(1, idx, (ws * inner * (1.0 - s_sel)).masked_fill(none, 0.0))
        else:
            dx = dx.scatter_add(1, idx, (dw * s_sel * (1.0 - s_sel)).masked_fill(none, 0.0))
    out["dlogits"] = dx.to(st["logits"].dtype)
    return out


def _plain_dispatch(st):
    c = st["case"]
    T, K = st["idx"].shape
    E = c["E"]
    e = st["idx"].flatten().long()
    key = torch.where(e < 0, E, e)
    srt = torch.sort(key, stable=True)
    off = (srt.values.unsqueeze(0) < torch.arange(E + 1, device=e.device).unsqueeze(1)).sum(1)
    pair = torch.arange(T * K, device=e.device)
    rows = torch.empty_like(pair)
    rows[srt.indices] = pair
    return {"expert_off": off.int(),
            "row_index": torch.where(srt.values < E, srt.indices // K, -1).int(),
            "row_of": torch.where(e < 0, -1, rows).int().view(T, K)}


def _dequant(q, sc):
    R, C = q.shape
    v = q.view(torch.float8_e4m3fn).float().view(R, C // 32, 32)
    return torch.ldexp(v, (sc.int() - 127).unsqueeze(2)).view(R, C)


def _erf_cdf(x):
    return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, 0.0)
    if name == "gelu":
        return z * _erf_cdf(z)
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    F = z.shape[1] // 2
    gate, up = z[:, :F], z[:, F:]
    return _act("silu" if name == "swiglu" else "gelu", gate) * up


def _act_slope(name, z):
    if name == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if name == "gelu":
        return _erf_cdf(z) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def _plain_ffn(st):
    c = st["case"]
    E, N, Kd, M = c["E"], c["N"], c["Kd"], c["M"]
    out_f = N // 2 if c["act"] in GATED else N
    y = torch.empty(M, out_f, dtype=torch.bfloat16, device=DEV)
    z = torch.empty(M, N, dtype=torch.bfloat16, device=DEV) if c["save"] else None
    xs = _from_atoms(st["xs"], st["xq"].shape[0], Kd)
    ws = _from_atoms(st["ws"], st["wq"].shape[0], Kd)
    p = r = 0
    for e, n in enumerate(st["counts"]):
        if n:
            a = _dequant(st["xq"][p:p + n], xs[p:p + n])
            b = _dequant(st["wq"][e * N:(e + 1) * N], ws[e * N:(e + 1) * N])
            v = a @ b.T
            if st["bias"] is not None:
                v = v + st["bias"][e]
            if z is not None:
                z[r:r + n] = v.bfloat16()
            h = _act(c["act"], v)
            if st["residual"] is not None:
                h = h + st["residual"][r:r + n].float()
            y[r:r + n] = h.bfloat16()
        p += (n + 127) // 128 * 128
        r += n
    return {"y": y, "preact": z} if c["save"] else {"y": y}


def _plain_act(st):
    c = st["case"]
    z, dy = st["z"].float(), st["dy"].float()
    if c["act"] in GATED:
        F = c["N"] // 2
        inner = "silu" if c["act"] == "swiglu" else "gelu"
        gate, up = z[:, :F], z[:, F:]
        dz = torch.cat([dy * up * _act_slope(inner, gate), dy * _act(inner, gate)], 1)
    else:
        dz = dy * _act_slope(c["act"], z)
    out = {"dz": dz.bfloat16()}
    if c["bias"]:
        db = torch.zeros(c["E"], c["N"], device=DEV)
        r = 0
        for e, n in enumerate(st["counts"]):
            db[e] = dz[r:r + n].sum(0)
            r += n
        out["dbias"] = db
    return out


def _plain_combine(st):
    c = st["case"]
    T, K, H = c["T"], c["K"], c["H"]
    y, w, rows = st["y"], st["weights"], st["row_of"].long()
    acc = torch.zeros(T, H, device=DEV)
    if st["residual"] is not None:
        acc = st["residual"].float()
    safe = rows.clamp(min=0)
    wz = w.masked_fill(rows < 0, 0.0)
    if y.shape[0] > 0:
        for k in range(K):
            acc = acc + wz[:, k:k + 1] * y[safe[:, k]].float()
    out = {"out": acc.to(y.dtype)}
    if c["train"]:
        d = st["dout"].float()
        dy = torch.zeros_like(y)
        dw = torch.zeros(T, K, device=DEV)
        for k in range(K):
            has = (rows[:, k] >= 0).nonzero().flatten()
            dy[rows[has, k]] = (w[has, k:k + 1] * d[has]).to(y.dtype)
            dw[has, k] = (d[has] * y[rows[has, k]].float()).sum(1)
        out["dy"], out["dweights"] = dy, dw
    return out


# -------------------------------------------------------------------------- the library's calls
def _own(st):
    from moe_grouped_gemm_wgrad_gb300 import mgw
    c = st["case"]
    op = c["op"]
    if op == "route":
        score = mgw.SCORE_SOFTMAX if c["score"] == "softmax" else mgw.SCORE_SIGMOID
        r = mgw.moe_route(st["logits"], c["K"], bias=st["bias"], score=score, groups=c["groups"],
                          top_groups=c["top_groups"], group_best=1 if st["bias"] is None else 2,
                          renorm=c["renorm"], scale=c["scale"], with_scores=c["train"])
        out = {"expert_idx": r[0], "weights": r[1]}
        if c["train"]:
            out["scores"] = r[2]
            out["dlogits"] = mgw.moe_route_backward(st["logits"], r[0], st["dweights"],
                                                    dscores=st["dscores"], score=score,
                                                    renorm=c["renorm"], scale=c["scale"])
        return out
    if op == "dispatch":
        off, row_index, row_of = mgw.moe_dispatch(st["idx"], c["E"])
        return {"expert_off": off, "row_index": row_index, "row_of": row_of}
    if op in ("ffn", "act"):
        act = {"none": mgw.ACT_NONE, "relu": mgw.ACT_RELU, "gelu": mgw.ACT_GELU,
               "silu": mgw.ACT_SILU, "swiglu": mgw.ACT_SWIGLU, "geglu": mgw.ACT_GEGLU}[c["act"]]
        if op == "ffn":
            r = mgw.grouped_fprop_mxfp8_act(st["xq"], st["xs"], st["wq"], st["ws"], st["off"],
                                            c["M"], c["N"], act, bias=st["bias"],
                                            residual=st["residual"], save_preact=c["save"])
            return {"y": r[0], "preact": r[1]} if c["save"] else {"y": r}
        dz, db = mgw.grouped_act_backward(st["dy"], st["z"], st["off"], act, with_dbias=c["bias"])
        return {"dz": dz, "dbias": db} if c["bias"] else {"dz": dz}
    out = {"out": mgw.moe_combine(st["y"], st["row_of"], weights=st["weights"],
                                  residual=st["residual"])}
    if c["train"]:
        out["dy"], out["dweights"] = mgw.moe_combine_backward(st["dout"], st["y"], st["row_of"],
                                                              weights=st["weights"])
    return out


def run(state):
    if own:
        return _own(state)
    return {"route": _plain_route, "dispatch": _plain_dispatch, "ffn": _plain_ffn,
            "act": _plain_act, "combine": _plain_combine}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- work
def work(case):
    c = case
    op = c["op"]
    if op == "route":
        T, E, K = c["T"], c["E"], c["K"]
        el = 2 if c["dtype"] == "bf16" else 4
        b = T * E * el + T * K * 8 + (4 * E if c["bias"] else 0)
        f = 4 * T * E
        if c["train"]:
            b += T * E * 4 + T * K * 4 + T * E * 4 + T * E * el  # scores, dweights, dscores, dlogits
            f += 6 * T * E
        return {"bytes": b, "flops": f}
    if op == "dispatch":
        pairs = c["T"] * min(c["K"], c["E"])
        return {"bytes": 12 * pairs + 4 * (c["E"] + 1), "flops": pairs}
    if op in ("ffn", "act"):
        M, E, N = c["M"], c["E"], c["N"]
        out_f = N // 2 if c["act"] in GATED else N
        if op == "act":
            return {"bytes": 2 * M * N * 2 + 2 * M * out_f + 4 * (E + 1) + (4 * E * N if c["bias"] else 0),
                    "flops": 10 * M * N}
        Kd = c["Kd"]
        used = min(E, M)  # experts that have rows
        b = (M + used * N) * (Kd + Kd // 32) + 2 * M * out_f + 4 * (E + 1)
        b += (4 * used * N if c["bias"] else 0) + (2 * M * out_f if c["residual"] else 0)
        b += 2 * M * N if c["save"] else 0
        return {"bytes": b, "flops": 2 * M * N * Kd}
    T, K, H = c["T"], c["K"], c["H"]
    el = 2 if c["dtype"] == "bf16" else 4
    M = int(T * K * (1 - c["dropped"]))
    b = M * H * el + T * H * el + T * K * 8 + (T * H * el if c["residual"] else 0)
    f = 2 * M * H
    if c["train"]:
        b += T * H * el + M * H * el + T * K * 4  # dout, dy, dweights
        f += 3 * M * H
    return {"bytes": b, "flops": f}


# ------------------------------------------------------------------------- 64-bit definitions
def _exact_route(c, st):
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    x = st["logits"].double()
    usable = x > NEG
    alive = usable.any(1, keepdim=True)
    filled = torch.where(alive, x, torch.zeros_like(x))
    s = torch.softmax(filled, 1) if c["score"] == "softmax" else torch.sigmoid(filled)
    s = torch.where(usable, s, torch.zeros_like(s))
    rank_by = x if st["bias"] is None else torch.where(usable, s + st["bias"].double(), NEG)
    allowed = usable
    if G > 1:
        per = torch.sort(rank_by.view(T, G, -1), 2, descending=True).values
        gs = per[:, :, 0].clone()
        if st["bias"] is not None and per.shape[2] > 1:
            second = per[:, :, 1]
            gs = torch.where(second > NEG, gs + second, gs)
        order = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        kept = torch.zeros(T, G, device=x.device).scatter(1, order, 1.0) > 0
        allowed = allowed & kept.unsqueeze(2).expand(T, G, E // G).reshape(T, E)
    srt = torch.sort(torch.where(allowed, rank_by, NEG), dim=1, descending=True, stable=True)
    idx, real = srt.indices[:, :K], srt.values[:, :K] > NEG
    raw = torch.where(real, torch.gather(s, 1, idx), 0.0)
    if c["renorm"]:
        if c["score"] == "softmax":
            lw = torch.where(real, torch.gather(x, 1, idx), NEG)
            share = torch.nan_to_num(torch.softmax(lw, 1), nan=0.0)
        else:
            tot = raw.sum(1, keepdim=True)
            share = raw / torch.where(tot > 0, tot, 1.0)
    else:
        share = raw
    out = {"expert_idx": torch.where(real, idx, -1).int(), "weights": c["scale"] * share}
    if c["train"]:
        out["scores"] = s
        # the gradient through a dense Jacobian product: G = dL/dscores, then through the score
        dw = torch.where(real, st["dweights"].double() * c["scale"], 0.0)
        grad = torch.where(usable, st["dscores"].double(), 0.0)
        if c["renorm"]:
            tot = raw.sum(1, keepdim=True)
            tot = torch.where(tot > 0, tot, 1.0)
            dsel = (dw - (dw * share).sum(1, keepdim=True)) / tot
        else:
            dsel = dw
        grad = grad.scatter_add(1, idx, torch.where(real, dsel, 0.0))
        if c["score"] == "softmax":
            out["dlogits"] = s * (grad - (grad * s).sum(1, keepdim=True))
        else:
            out["dlogits"] = grad * s * (1 - s)
    return out


def _exact_dispatch(c, st):
    T, K = st["idx"].shape
    E = c["E"]
    e = st["idx"].flatten().cpu().tolist()
    lists = [[] for _ in range(E)]
    for i, ex in enumerate(e):
        if ex >= 0:
            lists[ex].append(i)
    off, order = [0], []
    for li in lists:
        order += li
        off.append(len(order))
    row_of = [-1] * (T * K)
    for r, i in enumerate(order):
        row_of[i] = r
    rows = [i // K for i in order] + [-1] * (T * K - len(order))
    i32 = {"dtype": torch.int32, "device": DEV}
    return {"expert_off": torch.tensor(off, **i32), "row_index": torch.tensor(rows, **i32),
            "row_of": torch.tensor(row_of, **i32).view(T, K)}


def _phi(x):
    return 0.5 * torch.erfc(-x / math.sqrt(2.0))


def _exact_ffn(c, st):
    E, N, Kd, act = c["E"], c["N"], c["Kd"], c["act"]
    f8 = torch.arange(256, device=DEV, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()

    def values(q, atoms, r0, n):
        """Rows r0 .. r0+n of an operand: each element's value times its block's scale."""
        r = torch.arange(r0, r0 + n, device=DEV).unsqueeze(1)
        b = torch.arange(Kd // 32, device=DEV).unsqueeze(0)
        at = ((b // 4) * (q.shape[0] // 128) + r // 128) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
        sc = torch.pow(2.0, atoms[at].double() - 127.0)
        return f8[q[r0:r0 + n].int()] * sc.repeat_interleave(32, 1)

    ys, zs = [], []
    p = r = 0
    for e in range(E):
        n = st["counts"][e]
        if n:
            v = values(st["xq"], st["xs"], p, n) @ values(st["wq"], st["ws"], e * N, N).T
            if c["bias"]:
                v += st["bias"][e].double()
            gate = v[:, :N // 2] if act in GATED else v
            if act in ("gelu", "geglu"):
                h = gate * _phi(gate)
            elif act in ("silu", "swiglu"):
                h = gate * torch.sigmoid(gate)
            elif act == "relu":
                h = torch.clamp(gate, min=0.0)
            else:
                h = gate
            if act in GATED:
                h = h * v[:, N // 2:]
            if c["residual"]:
                h = h + st["residual"][r:r + n].double()
            ys.append(h)
            zs.append(v)
        p += -(-n // 128) * 128
        r += n
    out = {"y": torch.cat(ys)}
    if c["save"]:
        out["preact"] = torch.cat(zs)
    return out


def _exact_act(c, st):
    z, dy, act = st["z"].double(), st["dy"].double(), c["act"]
    gate = z[:, :c["N"] // 2] if act in GATED else z
    if act in ("gelu", "geglu"):
        cdf = _phi(gate)
        slope = cdf + gate * torch.exp(-gate ** 2 / 2) / math.sqrt(2 * math.pi)
        val = gate * cdf
    elif act in ("silu", "swiglu"):
        sg = torch.sigmoid(gate)
        slope = sg + gate * sg * torch.sigmoid(-gate)
        val = gate * sg
    else:
        slope, val = (gate > 0).double(), None
    dz = dy * slope if act not in GATED else torch.cat([dy * z[:, c["N"] // 2:] * slope, dy * val], 1)
    out = {"dz": dz}
    if c["bias"]:
        e = torch.repeat_interleave(torch.arange(c["E"], device=DEV),
                                    torch.tensor(st["counts"], device=DEV))
        out["dbias"] = torch.zeros(c["E"], c["N"], dtype=torch.float64, device=DEV).index_add_(0, e, dz)
    return out


def _exact_combine(c, st):
    T, K, H = c["T"], c["K"], c["H"]
    y, w, rows = st["y"].double(), st["weights"].double(), st["row_of"].long()
    token = torch.arange(T, device=DEV).unsqueeze(1).expand(T, K)
    named = rows >= 0
    src, dst, wt = rows[named], token[named], w[named].unsqueeze(1)
    out = st["residual"].double() if c["residual"] else torch.zeros(T, H, dtype=torch.float64, device=DEV)
    res = {"out": out.index_add(0, dst, wt * y[src])}
    if c["train"]:
        d = st["dout"].double()
        dy = torch.zeros_like(y)
        dy[src] = wt * d[dst]
        dw = torch.zeros(T, K, dtype=torch.float64, device=DEV)
        dw[named] = torch.einsum("rh,rh->r", d[dst], y[src])
        res["dy"], res["dweights"] = dy, dw
    return res


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "dispatch": _exact_dispatch, "ffn": _exact_ffn,
            "act": _exact_act, "combine": _exact_combine}[case["op"]](case, st)
