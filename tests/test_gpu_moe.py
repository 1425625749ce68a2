"""The routed-layer operators on the GPU against 64-bit restatements.

Tolerances, from the arithmetic:
* router weights and scores (fp32): an exponential is good to 2 ulp, its argument x - m of
  size up to 32 is rounded to 2^-24 of itself (2e-6 at 32, typically far less), the sum and the
  division add 1 ulp each: |error| <= 4e-6 of the value.
* dlogits: a sum of products of such values, so 1e-5 of the largest term of its row, plus half
  an ulp of the output's type (2^-9 of the value for bf16).
* the expert product: fp32 accumulation of exact products; the accumulator's error is far below
  bf16's half ulp, 2^-9 = 2e-3 of the value.  An activation moves its argument's error by a
  slope of at most 1.13 and gated ones multiply two values: 4e-3 |y| + 1e-3 rms(y).
* combine: fp32 sum of <= 9 terms: 1e-6 of the sum of magnitudes, plus the output's half ulp.
* dweights, dbias: fp32 sums of n terms in blocks: 2^-24 * (n / 8 + 16) of the sum of magnitudes,
  a bound on any order that is at most n / 8 + 16 additions deep.
"""
import numpy as np
import pytest
import torch

import moe_reference as ref
import oracle
from moe_grouped_gemm_wgrad_gb300 import mgw, synth
from helpers import dev_bf16, dev_i32

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SCORE = {"softmax": mgw.SCORE_SOFTMAX, "sigmoid": mgw.SCORE_SIGMOID}
ACT = {"none": mgw.ACT_NONE, "relu": mgw.ACT_RELU, "gelu": mgw.ACT_GELU, "silu": mgw.ACT_SILU,
       "swiglu": mgw.ACT_SWIGLU, "geglu": mgw.ACT_GEGLU}
GATED = ("swiglu", "geglu")
HALF_ULP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -23}


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(DT[dtype])


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------------- router
def _logits(rng, T, E, dtype, masked):
    x = rng.standard_normal((T, E)) * 1.5
    if dtype == "bf16":
        x = ref.bf16(x)                 # bf16 logits tie often
    else:
        x = np.float32(x).astype(np.float64)
    if masked:
        x[rng.random((T, E)) < masked] = ref.NEG
        x[rng.random(T) < 0.1] = ref.NEG
    return x


ROUTES = [
    # T, E, K, dtype, score, bias, groups, top_groups, group_best, renorm, scale, masked
    (1, 8, 1, "bf16", "softmax", False, 1, 1, 1, True, 1.0, 0),
    (1, 1, 1, "f32", "sigmoid", False, 1, 1, 1, True, 1.0, 0),
    (33, 64, 8, "bf16", "softmax", False, 1, 1, 1, True, 1.0, 0),
    (100, 61, 6, "bf16", "softmax", False, 1, 1, 1, False, 2.5, 0.3),
    (57, 32, 32, "f32", "softmax", False, 1, 1, 1, True, 1.0, 0.5),
    (40, 33, 4, "bf16", "sigmoid", False, 1, 1, 1, True, 1.0, 0.2),
    (64, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5, 0),
    (64, 256, 8, "f32", "sigmoid", True, 8, 4, 2, True, 2.5, 0.6),
    (31, 160, 6, "bf16", "softmax", False, 8, 3, 1, False, 16.0, 0.1),
    (31, 110, 5, "f32", "softmax", False, 2, 1, 2, True, 1.0, 0.1),
    (17, 512, 10, "bf16", "softmax", True, 1, 1, 1, False, 1.0, 0.05),
    (9, 1024, 16, "bf16", "sigmoid", True, 32, 5, 2, True, 1.0, 0.05),
    (9, 1000, 3, "f32", "softmax", False, 4, 2, 1, True, 1.0, 0),
    (25, 96, 8, "bf16", "softmax", False, 32, 3, 1, True, 1.0, 0),
    (12, 129, 7, "f32", "sigmoid", True, 3, 3, 2, False, 1.0, 0),
    # groups that cut across a lane's experts, with two and four tokens to a warp
    (67, 12, 1, "bf16", "softmax", False, 4, 1, 1, True, 2.5, 0),
    (66, 60, 5, "f32", "sigmoid", True, 20, 7, 2, True, 1.0, 0.2),
    (35, 96, 12, "bf16", "softmax", False, 32, 9, 1, True, 1.0, 0.3),
    (35, 126, 3, "f32", "softmax", True, 2, 1, 2, False, 1.0, 0.1),
    (37, 263, 11, "bf16", "softmax", False, 1, 1, 1, False, 1.0, 0.2),
    (5, 777, 4, "f32", "sigmoid", True, 7, 2, 2, True, 1.0, 0.1),
    # four, eight and sixteen lanes to a token, with one choice a lane and with two
    (41, 8, 2, "bf16", "softmax", False, 1, 1, 1, True, 1.0, 0.1),
    (70, 32, 8, "f32", "sigmoid", True, 1, 1, 1, True, 2.5, 0.2),
    (39, 31, 5, "bf16", "softmax", False, 1, 1, 1, False, 1.0, 0.1),
    (63, 32, 6, "f32", "softmax", True, 4, 2, 2, True, 1.0, 0.2),
    (63, 32, 3, "bf16", "sigmoid", False, 2, 1, 1, False, 1.0, 0.1),
    (50, 24, 7, "bf16", "sigmoid", True, 8, 5, 2, True, 1.0, 0.2),
    (44, 28, 10, "bf16", "sigmoid", True, 2, 2, 1, True, 1.0, 0.1),
    (37, 64, 16, "f32", "softmax", False, 8, 4, 1, True, 1.0, 0.1),
    (37, 61, 9, "bf16", "softmax", False, 1, 1, 1, False, 2.5, 0.9),
    (21, 128, 32, "bf16", "softmax", False, 1, 1, 1, True, 1.0, 0.1),
    (21, 100, 17, "f32", "sigmoid", False, 4, 3, 1, True, 1.0, 0.5),
    (19, 9, 9, "f32", "softmax", True, 1, 1, 1, False, 1.0, 0.3),
]


@pytest.mark.parametrize("T,E,K,dtype,score,bias,groups,top_groups,best,renorm,scale,masked", ROUTES)
def test_route(T, E, K, dtype, score, bias, groups, top_groups, best, renorm, scale, masked):
    rng = np.random.default_rng(T * 1000 + E)
    x = _logits(rng, T, E, dtype, masked)
    b = np.float32(np.round(rng.standard_normal(E) * 40) * 1e-3) if bias else None
    st = status()
    idx, w, s = mgw.moe_route(dev(x, dtype), K, bias=None if b is None else dev(b, "f32"),
                              score=SCORE[score], groups=groups, top_groups=top_groups,
                              group_best=best, renorm=renorm, scale=scale, with_scores=True,
                              status=st)
    assert st.item() == 0
    idx, w, s = idx.cpu().numpy(), f64(w), f64(s)
    judged = 0
    for t in range(T):
        want = ref.route_scores(x[t], score)
        assert np.all(np.abs(s[t] - want) <= 4e-6 * want + 1e-37), t
        e, wt, gap = ref.route_token(x[t], K, b, score, groups, top_groups, best, renorm, scale)
        # With sums of rounded scores, values closer than their rounding may go either way.
        # Comparisons of the logits themselves are exact, ties included.
        rounded = bias or (groups > top_groups and best == 2)
        if rounded and gap < 2e-6:
            continue
        judged += 1
        assert idx[t].tolist() == e, t
        assert np.all(np.abs(w[t] - wt) <= 4e-6 * np.abs(wt) + 1e-37), t
    assert judged >= 0.8 * T


def test_route_extreme_logits():
    low = float(torch.finfo(torch.bfloat16).min)
    inf = np.inf
    x = np.array([[low] * 8, [low] * 7 + [0.0], [-inf] * 8, [inf, 0, inf, 1, 2, 3, 4, 5],
                  [-inf] * 7 + [3.0], [0.0, -0.0, 0.0, -0.0, 0.0, 0.0, 0.0, 0.0],
                  [88.0, -88.0, 120.0, -120.0, 0, 0, 0, 0]])
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            st = status()
            idx, w, s = mgw.moe_route(dev(x, "bf16"), 3, score=SCORE[score], renorm=renorm,
                                      with_scores=True, status=st)
            idx, w, s = idx.cpu().numpy(), f64(w), f64(s)
            assert st.item() == 0 and np.isfinite(w).all() and np.isfinite(s).all()
            assert idx[0].tolist() == [0, 1, 2]          # a row of the type's lowest value: a tie
            assert idx[1].tolist() == [7, 0, 1]
            assert idx[2].tolist() == [-1, -1, -1] and (w[2] == 0).all() and (s[2] == 0).all()
            assert idx[3].tolist() == [0, 2, 7]
            assert idx[4].tolist() == [7, -1, -1] and (w[4][1:] == 0).all()
            assert idx[5].tolist() == [0, 1, 2]          # both zeros are one value
            if score == "softmax":
                assert np.allclose(w[0], 1 / 3 if renorm else 1 / 8, rtol=4e-6)
                assert np.allclose(w[1], [1, 0, 0]) and np.allclose(w[3], [0.5, 0.5, 0])
                assert w[4][0] == 1.0
            assert idx[6].tolist() == [2, 0, 4]


def test_route_renormalised_logistic_scores_that_underflow():
    """Renormalised logistic weights s_k / sum s where every s is below fp32's (and the last rows
    below 64 bits') range: s = e^x / (1 + e^x), and e^x may be taken out of the quotient."""
    rows = [[-89.0, -89.5, -90.25, -300.0], [-100.0, -101.0, -103.5, -120.0], [-150.0, -151.0, -150.5, -400.0],
            [-1000.0, -1001.0, -1000.25, -2000.0], [-3.0e38, -3.0e38, -3.2e38, -3.3e38], [2.0, -1.0, -90.0, -200.0]]
    x = np.array(rows)
    idx, w = mgw.moe_route(dev(x, "f32"), 3, score=SCORE["sigmoid"], scale=2.5)
    idx, w = idx.cpu().numpy(), f64(w)
    x = np.float32(x).astype(np.float64)
    g = np.float32(np.random.default_rng(3).standard_normal((len(x), 3)))
    d = f64(mgw.moe_route_backward(dev(x, "f32"), dev_i32(idx), dev(g, "f32"), score=SCORE["sigmoid"], scale=2.5))
    for t in range(len(x)):
        assert sorted(idx[t]) == [0, 1, 2], t
        xk = x[t][idx[t]]
        up = np.exp(np.maximum(xk, -700)) * (xk > -700)
        p = np.exp(np.maximum(xk - xk.max(), -700)) / (1 + up)
        p /= p.sum()
        assert np.all(np.abs(w[t] - 2.5 * p) <= 4e-6 * 2.5 * p + 1e-37), t
        want = np.zeros(4)
        want[idx[t]] = 2.5 * p * (g[t] - (p * g[t]).sum()) / (1 + up)
        assert np.all(np.abs(d[t] - want) <= 1e-5 * 2.5 * np.abs(g[t]).max()), t


def test_route_reports_a_logit_that_is_not_a_number():
    x = torch.zeros(3, 16, device="cuda")
    x[1, 5] = float("nan")
    x[1, 6] = 1.0
    st = status()
    idx, w = mgw.moe_route(x, 2, status=st)
    assert st.item() == mgw.MGW_DEV_BAD_LOGIT
    assert idx.tolist() == [[0, 1], [6, 0], [0, 1]] and torch.isfinite(w).all()


def test_route_no_tokens_and_given_buffers():
    idx, w = mgw.moe_route(torch.empty(0, 16, device="cuda"), 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    x = torch.randn(5, 16, device="cuda")
    bi, bw = torch.empty(5, 2, dtype=torch.int32, device="cuda"), torch.empty(5, 2, device="cuda")
    idx, w = mgw.moe_route(x, 2, expert_idx=bi, weights=bw)
    assert idx is bi and w is bw
    assert idx.long().tolist() == torch.topk(x, 2).indices.tolist()


def test_route_offsets_past_32_bits():
    """The last tokens of a logits matrix with more than 2^31 elements."""
    T, E = (1 << 21) + 64, 1024
    x = torch.zeros(T, E, dtype=torch.bfloat16, device="cuda")
    pick = torch.arange(T - 50, T, device="cuda")
    x[pick, pick % E] = 4.0
    idx, _ = mgw.moe_route(x, 1)
    assert idx[-50:, 0].tolist() == (pick % E).tolist() and int(idx[:-50].abs().max()) == 0
    d = mgw.moe_route_backward(x, idx, torch.ones(T, 1, device="cuda"), renorm=False)
    want = ref.route_backward_token(f64(x[-1]), [int(idx[-1, 0])], [1.0], None, "softmax", False, 1.0)
    assert np.all(np.abs(f64(d[-1]) - want) <= 2.0 ** -8 * np.abs(want) + 1e-5 * np.abs(want).max())


@pytest.mark.parametrize("T,E,K,dtype,score,renorm,masked,dw,ds", [
    (1, 8, 2, "f32", "softmax", True, 0, True, False),
    (33, 64, 8, "bf16", "softmax", False, 0, True, True),
    (20, 64, 8, "bf16", "softmax", True, 0.3, True, True),
    (20, 61, 4, "f32", "softmax", False, 0.3, True, False),
    (20, 256, 8, "f32", "sigmoid", True, 0.2, True, False),
    (20, 110, 5, "bf16", "sigmoid", False, 0.2, True, True),
    (7, 1000, 9, "f32", "softmax", True, 0, True, True),
    (7, 512, 32, "f32", "sigmoid", True, 0.9, True, True),
    (9, 40, 3, "f32", "softmax", True, 0, False, True),
    (37, 263, 11, "bf16", "softmax", False, 0.2, True, True),
    (70, 12, 2, "bf16", "sigmoid", True, 0.2, True, True),
    (33, 101, 9, "f32", "softmax", False, 0.1, True, True),
    (6, 777, 30, "f32", "sigmoid", False, 0.1, True, True),
    (9, 40, 3, "f32", "sigmoid", True, 0, False, False),
    (45, 28, 10, "bf16", "sigmoid", True, 0.1, True, True), (37, 20, 8, "f32", "softmax", True, 0.2, True, True),
    (19, 128, 32, "f32", "softmax", True, 0, True, False), (23, 64, 13, "f32", "sigmoid", False, 0, True, False),
    (66, 8, 5, "bf16", "softmax", False, 0.1, True, True), (17, 100, 17, "f32", "sigmoid", True, 0, True, True),
])
def test_route_backward(T, E, K, dtype, score, renorm, masked, dw, ds):
    rng = np.random.default_rng(T + E * 7)
    x = _logits(rng, T, E, dtype, masked)
    gw = np.float32(rng.standard_normal((T, K))) if dw else None
    gs = np.float32(rng.standard_normal((T, E))) if ds else None
    st = status()
    xd = dev(x, dtype)
    idx, _ = mgw.moe_route(xd, K, score=SCORE[score], renorm=renorm, scale=2.5, status=st)
    out = torch.full((T, E), float("nan"), dtype=DT[dtype], device="cuda")
    d = mgw.moe_route_backward(xd, idx, None if gw is None else dev(gw, "f32"),
                               dscores=None if gs is None else dev(gs, "f32"), score=SCORE[score],
                               renorm=renorm, scale=2.5, dlogits=out, status=st)
    assert st.item() == 0
    got, idx = f64(d), idx.cpu().numpy()
    for t in range(T):
        want = ref.route_backward_token(x[t], idx[t].tolist(), None if gw is None else gw[t],
                                        None if gs is None else gs[t], score, renorm, 2.5)
        big = 2.5 * (np.abs(gw[t]).max() if dw else 0) + (np.abs(gs[t]).max() if ds else 0)
        assert np.all(np.abs(got[t] - want) <= HALF_ULP[dtype] * np.abs(want) + 1e-5 * big), t
        assert np.all(got[t][x[t] == ref.NEG] == 0)
    if dw and not masked:
        # against differences of the 64-bit weights, along one random direction per token
        for t in range(min(T, 8)):
            v = rng.standard_normal(E)
            h = 1e-5

            def loss(z):
                a = (ref.route_weights(z, idx[t].tolist(), score, renorm, 2.5) * gw[t]).sum()
                return a + ((ref.route_scores(z, score) * gs[t]).sum() if ds else 0.0)

            diff = (loss(x[t] + h * v) - loss(x[t] - h * v)) / (2 * h)
            tol = (HALF_ULP[dtype] * np.abs(got[t]) + 1e-5 * big) @ np.abs(v) + 1e-7
            assert abs(diff - got[t] @ v) <= tol


def test_route_backward_bad_expert_is_reported():
    x = torch.randn(4, 16, device="cuda")
    idx = torch.tensor([[0, 1], [2, 16], [3, -2], [4, -1]], dtype=torch.int32, device="cuda")
    st = status()
    d = mgw.moe_route_backward(x, idx, torch.ones(4, 2, device="cuda"), renorm=False, status=st)
    assert st.item() == mgw.MGW_DEV_BAD_INDEX
    want = ref.route_backward_token(f64(x[1]), [2, -1], [1.0, 0.0], None, "softmax", False, 1.0)
    assert np.all(np.abs(f64(d[1]) - want) <= 1e-5)


# ----------------------------------------------------------------------------- dispatch
@pytest.mark.parametrize("T,K,E,drop,skew", [
    (0, 2, 4, 0, 0), (1, 1, 1, 0, 0), (1, 8, 64, 0, 0), (31, 1, 7, 0, 0), (33, 3, 5, 0.2, 0),
    (16, 8, 64, 0, 0), (1000, 2, 1024, 0, 0), (1024, 8, 64, 0, 1), (1025, 8, 64, 0.05, 1),
    (4096, 8, 512, 0, 0), (30000, 7, 600, 0.3, 1), (131071, 8, 64, 0, 1), (50000, 3, 2, 1.0, 0),
    (200000, 6, 3, 0, 0), (8192, 1, 1, 0, 0), (8193, 1, 1000, 0, 0), (4096, 1, 512, 0, 0), (4097, 1, 512, 0, 1),
    (1100000, 4, 40, 0.01, 1), (1100001, 3, 1024, 0, 0), (1100000, 8, 40, 0.01, 1),
    # around one CTA, clusters of 2 to 16 CTAs, and two launches; the last runs of CTAs empty
    (2048, 1, 64, 0, 0), (2049, 1, 64, 0, 1), (683, 3, 64, 0.2, 0), (16384, 1, 64, 0, 0), (5462, 3, 64, 0, 1),
    (4097, 8, 512, 0.1, 0), (8192, 8, 64, 0, 1), (8193, 8, 64, 0, 0), (512, 2, 513, 0, 0), (1025, 1, 1024, 0, 0),
    (8193, 1, 600, 0.1, 1), (4096, 8, 1024, 0, 0), (32769, 1, 1024, 0, 0), (32769, 1, 1, 0, 0),
])
def test_dispatch(T, K, E, drop, skew):
    rng = np.random.default_rng(T + K + E)
    p = (np.arange(E) + 1.0) ** -skew
    idx = rng.choice(E, size=(T, K), p=p / p.sum()).astype(np.int32)
    idx[rng.random((T, K)) < drop] = -1
    st = status()
    off, row_index, row_of = mgw.moe_dispatch(dev_i32(idx), E, status=st)
    woff, wri, wro = ref.dispatch(idx, E)
    assert st.item() == 0
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(row_index.cpu().numpy(), wri)
    assert np.array_equal(row_of.cpu().numpy(), wro)


@pytest.mark.parametrize("T", [40, 20000])
def test_dispatch_reports_experts_out_of_range(T):
    rng = np.random.default_rng(T)
    idx = rng.integers(0, 9, (T, 2)).astype(np.int32)
    bad = idx.copy()
    bad[3, 1], bad[T - 1, 0] = 9, -7
    st = status()
    off, row_index, row_of = mgw.moe_dispatch(dev_i32(bad), 9, status=st)
    assert st.item() == mgw.MGW_DEV_BAD_INDEX
    idx[3, 1] = idx[T - 1, 0] = -1
    woff, wri, wro = ref.dispatch(idx, 9)
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(row_index.cpu().numpy(), wri) and np.array_equal(row_of.cpu().numpy(), wro)


# ------------------------------------------------------------------------------ combine
def _tables(rng, T, K, drop):
    idx = rng.integers(0, 5, (T, K))
    idx[rng.random((T, K)) < drop] = -1
    off, _, row_of = ref.dispatch(idx, 5)
    return row_of.astype(np.int32), int(off[-1])


@pytest.mark.parametrize("T,K,H,dtype,drop,residual,weighted", [
    (1, 1, 1, "f32", 0, False, True), (1, 8, 4096, "bf16", 0, True, True),
    (16, 8, 1536, "bf16", 0, True, True), (7, 3, 8, "bf16", 0.3, False, True),
    (13, 2, 129, "bf16", 0.2, True, True), (200, 4, 1999, "f32", 0.05, True, True),
    (64, 8, 260, "f32", 0, False, False), (65, 32, 72, "bf16", 0.5, True, True),
    (5, 2, 64, "bf16", 1.0, True, True), (5, 2, 64, "bf16", 1.0, False, False),
    (0, 2, 64, "bf16", 0, False, True), (3, 5, 10000, "bf16", 0, True, True),
    (9, 9, 1002, "bf16", 0.1, True, True), (9, 10, 2052, "bf16", 0.1, False, True), (9, 2, 4102, "f32", 0, True, True),
    (33, 17, 515, "f32", 0.1, True, True), (5000, 3, 264, "bf16", 0.1, True, True),
    # rows between 16-byte boundaries: shorter than a block, around it, around 31 blocks, longer
    (5, 3, 1, "bf16", 0, True, True), (6, 2, 2, "bf16", 0.1, True, True), (7, 4, 7, "bf16", 0.2, False, True),
    (9, 5, 9, "bf16", 0, True, True), (8, 3, 3, "f32", 0.1, True, True), (11, 4, 241, "bf16", 0.1, True, True),
    (11, 6, 247, "bf16", 0.1, True, True), (10, 9, 249, "bf16", 0, True, True), (12, 2, 1985, "bf16", 0.1, True, True),
    (12, 2, 1991, "bf16", 0.1, False, True), (13, 3, 125, "f32", 0, True, True), (9, 2, 4001, "bf16", 0.3, True, True),
    (6, 3, 6, "bf16", 0, True, False), (40, 8, 3311, "bf16", 0.1, True, True),
])
def test_combine_and_backward(T, K, H, dtype, drop, residual, weighted):
    rng = np.random.default_rng(T + K * 31 + H)
    row_of, M = _tables(rng, T, K, drop)
    rnd = ref.bf16 if dtype == "bf16" else (lambda a: np.float32(a).astype(np.float64))
    y, res, dout = (rnd(rng.standard_normal(s)) for s in ((M, H), (T, H), (T, H)))
    w = np.float32(rng.random((T, K))) if weighted else None
    if drop:
        if weighted:
            w[row_of < 0] = np.nan   # weights of dropped pairs are not used
    st = status()
    yd, rd, wd = dev(y, dtype), dev_i32(row_of), None if w is None else dev(w, "f32")
    out = mgw.moe_combine(yd, rd, weights=wd, residual=dev(res, dtype) if residual else None, status=st)
    want = ref.combine(y, row_of, w, res if residual else None)
    mag = ref.combine(np.abs(y), row_of, w, np.abs(res) if residual else None)
    assert np.all(np.abs(f64(out) - want) <= HALF_ULP[dtype] * np.abs(want) + 1e-6 * mag)
    dy, dw = mgw.moe_combine_backward(dev(dout, dtype), yd if weighted else None, rd, weights=wd,
                                      M=M, status=st)
    assert st.item() == 0
    wdy, wdw = ref.combine_backward(dout, y, row_of, w, M)
    assert np.all(np.abs(f64(dy) - wdy) <= HALF_ULP[dtype] * np.abs(wdy))
    if not weighted:
        assert dw is None
        return
    _, mag = ref.combine_backward(np.abs(dout), np.abs(y), row_of, w, M)
    assert np.all(np.abs(f64(dw) - wdw) <= 2.0 ** -24 * (H / 8 + 16) * mag)
    assert np.all(f64(dw)[row_of < 0] == 0)
    # out is linear in y and in w: <dout, out(y + v) - out(y)> = <dy, v> exactly
    v = rng.standard_normal((M, H))
    lhs = (dout * (ref.combine(v, row_of, w, None))).sum()
    tol = (HALF_ULP[dtype] * np.abs(wdy) * np.abs(v)).sum() + 1e-9
    assert abs(lhs - (f64(dy) * v).sum()) <= tol


def test_combine_in_place_residual_and_gather_gradient():
    rng = np.random.default_rng(5)
    row_of, M = _tables(rng, 50, 4, 0)
    y = torch.randn(M, 256, device="cuda")
    w = torch.rand(50, 4, device="cuda")
    res = torch.randn(50, 256, device="cuda")
    want = mgw.moe_combine(y, dev_i32(row_of), weights=w, residual=res)
    got = mgw.moe_combine(y, dev_i32(row_of), weights=w, residual=res, out=res)
    assert got is res and torch.equal(got, want)
    for width in (255, 130):   # rows between 16-byte boundaries
        yo, ro = y[:, :width].contiguous(), dev(rng.standard_normal((50, width)), "f32")
        want = mgw.moe_combine(yo, dev_i32(row_of), weights=w, residual=ro)
        assert torch.equal(mgw.moe_combine(yo, dev_i32(row_of), weights=w, residual=ro, out=ro), want)


def test_combine_keeps_neighbouring_rows():
    """A row of an odd width is stored without touching the rows beside it, and values beside the
    matrices (NaN here) reach nothing."""
    H = 333
    base = torch.full((64 * H,), float("nan"), dtype=torch.bfloat16, device="cuda")
    y = base[:20 * H].view(20, H)
    y.copy_(dev(np.random.default_rng(9).standard_normal((20, H)), "bf16"))
    row_of = torch.tensor([[19, 0], [3, -1], [7, 11]], dtype=torch.int32, device="cuda")
    out = torch.full((5, H), 9.0, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    mgw.moe_combine(y, row_of, weights=w, out=out[:3])
    assert (out[3:] == 9).all() and torch.isfinite(out).all()
    dy = torch.full((20, H), 9.0, dtype=torch.bfloat16, device="cuda")
    _, dw = mgw.moe_combine_backward(torch.ones(3, H, dtype=torch.bfloat16, device="cuda"), y, row_of,
                                     weights=w, dy=dy)
    named = [0, 3, 7, 11, 19]
    assert (dy[named] == 1).all() and torch.isfinite(dw).all()
    assert (dy[[r for r in range(20) if r not in named]] == 9).all()


def test_combine_reports_rows_out_of_range():
    y = torch.ones(4, 64, device="cuda")
    row_of = torch.tensor([[0, 4], [1, -2], [2, -1]], dtype=torch.int32, device="cuda")
    st = status()
    out = mgw.moe_combine(y, row_of, status=st)
    assert st.item() == mgw.MGW_DEV_BAD_INDEX and (out == 1).all()
    st = status()
    dy = torch.zeros(4, 64, device="cuda")
    _, dw = mgw.moe_combine_backward(torch.ones(3, 64, device="cuda"), y, row_of,
                                     weights=torch.ones(3, 2, device="cuda"), dy=dy, status=st)
    assert st.item() == mgw.MGW_DEV_BAD_INDEX
    assert dw.tolist() == [[64.0, 0.0]] * 3 and (dy[:3] == 1).all() and (dy[3] == 0).all()


def test_combine_offsets_past_32_bits():
    """Rows that start past 2^31 elements."""
    H = 32768
    M = (1 << 31) // H + 40
    y = torch.zeros(M, H, dtype=torch.bfloat16, device="cuda")
    y[M - 3:] = 2.0
    row_of = torch.tensor([[M - 1, 0], [M - 2, M - 3]], dtype=torch.int32, device="cuda")
    out = mgw.moe_combine(y, row_of)
    assert (out[0] == 2).all() and (out[1] == 4).all()
    dy, dw = mgw.moe_combine_backward(torch.ones(2, H, dtype=torch.bfloat16, device="cuda"), y, row_of,
                                      weights=torch.tensor([[3.0, 5.0], [7.0, 9.0]], device="cuda"), dy=y.clone())
    assert dw.tolist() == [[2.0 * H, 0.0], [2.0 * H, 2.0 * H]]
    assert (dy[M - 1] == 3).all() and (dy[0] == 5).all() and (dy[M - 3] == 9).all()


# -------------------------------------------------------------- the product's epilogue
def _operands(rng, counts, N, K):
    """MXFP8 operands on the GPU and z = x W^T in float64 from the oracle's own quantization."""
    E, M = len(counts), sum(counts)
    off = synth.offsets_from_counts(np.asarray(counts))
    xb = synth.bf16_bits_from_f32(rng.standard_normal((M, K)).astype(np.float32))
    wb = synth.bf16_bits_from_f32((rng.standard_normal((E * N, K)) * K ** -0.5).astype(np.float32))
    w_off = np.arange(E + 1, dtype=np.int32) * N
    src = dev_bf16(xb) if M else torch.empty((0, K), dtype=torch.bfloat16, device="cuda")
    xq, xs = mgw.mxfp8_quantize_rows(src, dev_i32(off))
    wq, ws = mgw.mxfp8_quantize_rows(dev_bf16(wb), dev_i32(w_off))
    if M:
        oxq, oxs = oracle.mxfp8_quantize_rows(xb, off)
        owq, ows = oracle.mxfp8_quantize_rows(wb, w_off)
        z = oracle.grouped_fprop_mx(oxq, oxs, owq, ows, off, w_off, M)
    else:
        z = np.zeros((0, N))
    return (xq, xs, wq, ws), off, z


@pytest.mark.parametrize("counts,N,K,act,bias,residual,save", [
    ([1], 256, 128, "none", False, False, False),
    ([0, 1, 0], 256, 256, "gelu", True, True, True),
    ([207, 208, 209], 256, 384, "silu", True, False, True),
    ([15, 16, 17, 0, 31, 33], 512, 1024, "relu", True, True, True),
    ([130, 0, 70], 512, 640, "swiglu", True, True, True),
    ([1030], 256, 512, "geglu", False, False, True),
    ([416, 417, 96, 97], 768, 256, "swiglu", False, True, False),
    ([5, 300, 0, 0, 64, 111, 2, 1], 512, 128, "gelu", False, False, False),
    ([0, 0], 256, 128, "swiglu", True, False, True),
    ([1, 1, 1, 1] * 10, 256, 256, "geglu", True, False, False),
    # few rows and items: the contraction is split over a cluster's pairs
    ([1], 256, 1024, "none", False, False, False),
    ([64], 512, 1152, "gelu", True, True, True),
    ([16], 4096, 1024, "swiglu", True, True, True),
    ([0, 33, 0, 31], 256, 2048, "silu", True, True, True),
    ([17, 1, 15, 0, 0, 20], 512, 640, "geglu", True, False, True),
    ([2, 3, 4, 5, 6, 7, 8, 9], 768, 512, "relu", False, True, True),
    ([48], 1024, 4096, "swiglu", False, False, False),
    ([65], 256, 1024, "gelu", True, True, True),
    ([0, 0, 0], 256, 1024, "gelu", True, False, True),
])
def test_fprop_act(counts, N, K, act, bias, residual, save):
    rng = np.random.default_rng(sum(counts) + N + K)
    E, M = len(counts), sum(counts)
    ops, off, z = _operands(rng, counts, N, K)
    F = N // 2 if act in GATED else N
    b = np.float32(rng.standard_normal((E, N))) if bias else None
    res = ref.bf16(rng.standard_normal((M, F))) if residual else None
    if bias:
        z = z + np.repeat(b.astype(np.float64), counts, axis=0)
    want = ref.act(act, z) + (res if residual else 0.0)
    st = status()
    out = torch.full((M + 3, F), 77.0, dtype=torch.bfloat16, device="cuda")
    got = mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(off), M, N, ACT[act],
                                      bias=None if b is None else dev(b, "f32"),
                                      residual=None if res is None else dev(res, "bf16"),
                                      save_preact=save, out=out, status=st)
    assert st.item() == 0
    if save:
        got, zg = got
        assert np.all(np.abs(f64(zg) - z) <= 4e-3 * np.abs(z) + 1e-3 * np.sqrt(np.mean(z ** 2) if M else 0))
    rms = np.sqrt(np.mean(want ** 2)) if M else 0.0
    assert np.all(np.abs(f64(got[:M]) - want) <= 4e-3 * np.abs(want) + 1e-3 * rms)
    assert (got[M:] == 77).all()   # nothing past the last row is touched


def test_fprop_act_matches_the_plain_product():
    """Without bias, activation or residual: the same product as grouped_fprop_mxfp8."""
    rng = np.random.default_rng(11)
    ops, off, z = _operands(rng, [300, 0, 129], 512, 512)
    a = mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(off), 429, 512)
    b = mgw.grouped_fprop_mxfp8(*ops, dev_i32(off), 429, 512)
    assert np.all(np.abs(f64(a) - f64(b)) <= 2.0 ** -7 * np.abs(z) + 1e-4)


def test_fprop_act_split_is_repeatable():
    rng = np.random.default_rng(13)
    ops, off, _ = _operands(rng, [40], 512, 2048)
    first = mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(off), 40, 512, mgw.ACT_SWIGLU)
    for _ in range(5):
        assert torch.equal(first, mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(off), 40, 512, mgw.ACT_SWIGLU))


@pytest.mark.parametrize("K", [128, 1024])
def test_fprop_act_bad_offsets_leave_outputs_alone(K):
    rng = np.random.default_rng(12)
    ops, off, _ = _operands(rng, [20, 30], 256, K)
    for bad in ([0, 50, 40], [1, 30, 50], [0, 30, 49]):
        st = status()
        out = torch.full((50, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(bad), 50, 256, out=out, status=st)
        assert st.item() == mgw.MGW_DEV_BAD_OFFSETS and (out == 5).all()
        st = status()
        dz = torch.full((50, 256), 5.0, dtype=torch.bfloat16, device="cuda")
        db = torch.full((2, 256), 5.0, device="cuda")
        mgw.grouped_act_backward(out, out, dev_i32(bad), mgw.ACT_RELU, dz=dz, dbias=db, status=st)
        assert st.item() == mgw.MGW_DEV_BAD_OFFSETS and (dz == 5).all() and (db == 5).all()


@pytest.mark.parametrize("counts,N,act", [
    ([1], 128, "relu"), ([0, 3, 0], 256, "gelu"), ([127, 128, 129], 384, "silu"),
    ([300, 0, 50], 512, "swiglu"), ([20, 900], 768, "geglu"), ([64, 65], 256, "none"),
    ([0, 0], 256, "gelu"), ([2] * 50, 128, "silu"), ([3000], 256, "swiglu"),
])
def test_act_backward(counts, N, act):
    rng = np.random.default_rng(sum(counts) + N)
    E, M = len(counts), sum(counts)
    off = synth.offsets_from_counts(np.asarray(counts))
    F = N // 2 if act in GATED else N
    dy = ref.bf16(rng.standard_normal((M, F)))
    z = ref.bf16(rng.standard_normal((M, N)) * 2)
    if M:
        z[0, :8] = [0.0, -0.0, 30.0, -30.0, 1e-30, -1e-30, 80.0, -100.0]
    zt = None if act == "none" else dev(z, "bf16")
    st = status()
    dz, db = mgw.grouped_act_backward(dev(dy, "bf16"), zt, dev_i32(off), ACT[act], with_dbias=True,
                                      status=st)
    assert st.item() == 0
    want = ref.act_backward(act, dy, z)
    # a slope is good to a few fp32 ulp of 1, times the gradient that meets it
    grad = np.abs(ref.act_backward("none", dy, z)) if act not in GATED else \
        np.concatenate([np.abs(dy * z[:, F:]), np.abs(dy) * np.maximum(np.abs(z[:, :F]), 1)], axis=1)
    assert np.all(np.abs(f64(dz) - want) <= 2.0 ** -8 * np.abs(want) + 2e-6 * grad)
    db = f64(db)
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        n = counts[e]
        assert np.all(np.abs(db[e] - want[rows].sum(axis=0)) <=
                      2.0 ** -24 * (n / 8 + 16) * np.abs(want[rows]).sum(axis=0)
                      + 2e-6 * grad[rows].sum(axis=0))
    # without the bias gradient: the same dz
    dz2, none = mgw.grouped_act_backward(dev(dy, "bf16"), zt, dev_i32(off), ACT[act])
    assert none is None and torch.equal(dz2, dz)


# --------------------------------------------------------------------- repeats, streams
def _whole(rng_seed=3, stream=None):
    """Every operator once, chained as a layer chains them; returns all outputs."""
    T, E, K, H, N = 300, 16, 4, 256, 512
    rng = np.random.default_rng(rng_seed)
    hidden = dev_bf16(synth.bf16_bits_from_f32(rng.standard_normal((T, H)).astype(np.float32)))
    wb = dev_bf16(synth.bf16_bits_from_f32((rng.standard_normal((E * N, H)) / 16).astype(np.float32)))
    w_off = dev_i32(np.arange(E + 1) * N)
    logits = dev(rng.standard_normal((T, E)), "f32")
    dout = dev(rng.standard_normal((T, N // 2)), "bf16")
    torch.cuda.synchronize()
    kw = {"stream": stream}
    ctx = torch.cuda.stream(stream) if stream is not None else torch.cuda.stream(torch.cuda.current_stream())
    with ctx:
        idx, w = mgw.moe_route(logits, K, **kw)
        off, row_index, row_of = mgw.moe_dispatch(idx, E, **kw)
        xq, xs = mgw.mxfp8_quantize_rows(hidden, off, row_index=row_index, **kw)
        wq, ws = mgw.mxfp8_quantize_rows(wb, w_off, **kw)
        y, z = mgw.grouped_fprop_mxfp8_act(xq, xs, wq, ws, off, T * K, N, mgw.ACT_SWIGLU,
                                           save_preact=True, **kw)
        out = mgw.moe_combine(y, row_of, weights=w, **kw)
        dy, dw = mgw.moe_combine_backward(dout, y, row_of, weights=w, **kw)
        dz, db = mgw.grouped_act_backward(dy, z, off, mgw.ACT_SWIGLU, with_dbias=True, **kw)
        dl = mgw.moe_route_backward(logits, idx, dw, **kw)
    (stream or torch.cuda.current_stream()).synchronize()
    return [idx, w, off, row_index, row_of, y, z, out, dy, dw, dz, db, dl]


def test_results_do_not_vary_between_runs_or_streams():
    a = _whole()
    for other in (_whole(), _whole(stream=torch.cuda.Stream())):
        assert all(torch.equal(x, y) for x, y in zip(a, other))


def test_operators_can_be_captured_in_a_graph():
    T, E, K, H = 64, 16, 4, 128
    logits = torch.randn(T, E, device="cuda")
    y = torch.randn(T * K, H, device="cuda")
    mgw.moe_route(logits, K)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        idx, w = mgw.moe_route(logits, K)
        _, _, row_of = mgw.moe_dispatch(idx, E)
        out = mgw.moe_combine(y, row_of, weights=w)
    logits.copy_(torch.randn(T, E, device="cuda"))
    g.replay()
    torch.cuda.synchronize()
    idx2, w2 = mgw.moe_route(logits, K)
    _, _, row2 = mgw.moe_dispatch(idx2, E)
    assert torch.equal(idx, idx2) and torch.equal(row_of, row2)
    assert torch.equal(out, mgw.moe_combine(y, row2, weights=w2))


@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "swiglu", "geglu"])
def test_special_values_through_the_epilogue(act):
    """z = bias alone (x is zero): infinities and NaN come out as the activation defines them."""
    inf, nan = float("inf"), float("nan")
    N, F = 256, 128 if act in GATED else 256
    off = dev_i32([0, 3])
    ops = (torch.zeros(256, 128, dtype=torch.uint8, device="cuda"),
           torch.full((1024,), 127, dtype=torch.uint8, device="cuda"),
           torch.zeros(384, 128, dtype=torch.uint8, device="cuda"),
           torch.full((1536,), 127, dtype=torch.uint8, device="cuda"), off)
    bias = torch.ones(1, N, device="cuda")
    bias[0, :7] = torch.tensor([inf, -1e30, 1e30, nan, 0.0, -0.0, -100.0])
    y = mgw.grouped_fprop_mxfp8_act(*ops, 3, N, ACT[act], bias=bias).float().cpu()
    assert (torch.equal(y[0], y[1]) or torch.equal(y[0].isnan(), y[1].isnan())) and y.shape == (3, F)
    assert y[0, 0] == inf and y[0, 1] == 0 and y[0, 2] > 9e29 and torch.isnan(y[0, 3])
    assert y[0, 4] == 0 and y[0, 5] == 0 and abs(float(y[0, 6])) < 1e-30
    assert torch.isfinite(y[:, 7:]).all()


def test_side_stream_allocations_are_kept():
    """Outputs and workspaces allocated by a call on another stream are not reused before that
    stream is done: many short-lived results while a long queue runs on the side stream."""
    side = torch.cuda.Stream()
    idx = torch.randint(0, 32, (20000, 8), device="cuda", dtype=torch.int32)
    want = mgw.moe_dispatch(idx, 32)
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device="cuda")
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 1e-2
    got = [mgw.moe_dispatch(idx, 32, stream=side) for _ in range(4)]
    for _ in range(8):   # the current stream writes over whatever the allocator hands out
        torch.full((1 << 18,), -77, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
