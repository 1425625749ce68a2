"""More of the expert product's epilogue and its backward pass on the GPU: special values on the way
back, many work items a CTA pair, a residual that is the output, bias sums over long and skewed
experts, and dropped pairs through a whole layer.

Tolerances are those of test_gpu_moe.py, from the same arithmetic: bf16's half ulp is at most 2^-8
of a value; 4e-3 |y| + 1e-3 rms(y) for the product; 2^-24 (n / 8 + 16) of the sum of magnitudes for
a sum of n terms that is at most n / 8 + 16 additions deep, plus 2e-6 of each term for its slope.
Every input comes from a generator of its test's own."""
import numpy as np
import pytest
import torch

import moe_reference as ref
import oracle
from moe_grouped_gemm_wgrad_gb300 import mgw, synth
from helpers import dev_bf16, dev_i32, oracle_quantize_by_expert
from test_gpu_moe import ACT, GATED, dev, f64, status

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


# -------------------------------------------------------------- special values on the way back
@pytest.mark.parametrize("act", ["relu", "gelu", "silu", "swiglu", "geglu"])
def test_special_values_on_the_way_back(act):
    """Finite z of any size has the formula's slope; NaN comes back as NaN and reaches nothing but
    its own element and its expert's sum of the column."""
    N = 256
    F = 128 if act in GATED else 256
    z = torch.ones(5, N)
    z[1, :9] = torch.tensor([NAN, INF, -INF, 0.0, -0.0, 3.3e38, -3.3e38, 1e-38, -100.0])
    dy = torch.full((5, F), 2.0)
    st = status()
    dz, db = mgw.grouped_act_backward(dev(dy.numpy(), "bf16"), dev(z.numpy(), "bf16"), dev_i32([0, 3, 5]),
                                      ACT[act], with_dbias=True, status=st)
    dz, db = dz.double().cpu(), db.double().cpu()
    assert st.item() == 0
    assert torch.isnan(dz[1, 0]) and torch.isnan(db[0, 0])
    slope = dz[1, :F] / 2
    if act == "relu":
        assert slope[1] == 1 and slope[2] == 0
    else:
        assert torch.isnan(slope[1]) and torch.isnan(slope[2])
    half = 0.0 if act == "relu" else 0.5
    assert slope[3] == half and slope[4] == half and slope[5] == 1 and slope[6] == 0
    assert slope[7] == (1.0 if act == "relu" else 0.5) and abs(slope[8]) < 1e-30
    odd = [0, 1, 2] if act != "relu" else [0]
    if act in GATED:   # the up columns' gradient is the gate's activation
        inner = "silu" if act == "swiglu" else "gelu"
        up = dz[1, F:] / 2
        assert torch.isnan(up[0]) and up[1] == INF and up[5] == INF   # 2 * 3.3e38 overflows
        assert torch.isnan(up[2]) if inner == "silu" else up[2] == 0
        odd += [F, F + 1, F + 5] + ([F + 2] if inner == "silu" else [])
    keep = torch.ones(N, dtype=torch.bool)
    keep[odd] = False
    assert torch.isfinite(db[0, keep]).all() and torch.isfinite(db[1]).all()
    assert torch.isfinite(dz[:, keep]).all() and torch.isfinite(dz[[0, 2, 3, 4]]).all()


def test_an_up_value_that_is_not_a_number_reaches_the_gate_only():
    z = torch.ones(3, 256)
    z[1, 128 + 7] = NAN
    dz, _ = mgw.grouped_act_backward(dev(np.ones((3, 128)), "bf16"), dev(z.numpy(), "bf16"), dev_i32([0, 3]),
                                     mgw.ACT_SWIGLU)
    bad = torch.isnan(dz).nonzero().tolist()
    assert bad == [[1, 7]]


def test_gelu_and_its_slope_before_any_rounding_to_bf16():
    """One row an expert and dy = 1: dbias is the slope itself in fp32, and the up columns' dbias of the
    gated form the GELU's value.  Over every bf16 z up to 14.

    The tail's formula is good to 1.5e-7 / 2; its factors t and e to about 2^-22 of themselves with the
    approximate reciprocal and exponential, of a tail of at most 1/2 whose derivative by them is below
    1 (2.4e-7); e counts once more in x phi(x), of at most 0.25, where its argument's rounding adds
    x^2 2^-24 (0.6e-7): 5e-7 for the slope, 4e-7 max(|x|, 1) for the value."""
    from scipy.special import erfc

    bits = np.arange(0x4160 + 1, dtype=np.uint16)          # 0 .. 14
    every = np.concatenate([bits, bits | 0x8000]).view(np.int16)
    E, N = 1024, 128
    z = torch.from_numpy(np.resize(every, E * N)).view(torch.bfloat16).view(E, N).cuda()
    off, x = dev_i32(np.arange(E + 1)), f64(z)
    phi = 0.5 * erfc(-x / np.sqrt(2.0))
    one = torch.ones(E, N, dtype=torch.bfloat16, device="cuda")
    _, db = mgw.grouped_act_backward(one, z, off, mgw.ACT_GELU, with_dbias=True)
    assert np.abs(f64(db) - (phi + x * np.exp(-x * x / 2) / np.sqrt(2 * np.pi))).max() <= 5e-7
    both = torch.cat([z, torch.ones_like(z)], dim=1)
    _, db = mgw.grouped_act_backward(one, both, off, mgw.ACT_GEGLU, with_dbias=True)
    assert (np.abs(f64(db)[:, N:] - x * phi) / np.maximum(np.abs(x), 1)).max() <= 4e-7


# ------------------------------------------------------------- many work items a CTA pair
MIXED = [33, 209, 1, 417, 150, 16, 0, 40]     # 1 to 3 row tiles of 1 to 13 groups of 16 rows


def _large_operands(rng, counts, N, K, product=True):
    """_operands for larger sizes: experts quantized on threads, z by matrix products in float64."""
    E, M = len(counts), sum(counts)
    off = synth.offsets_from_counts(np.asarray(counts))
    w_off = np.arange(E + 1, dtype=np.int32) * N
    xb = synth.bf16_bits_from_f32(rng.standard_normal((M, K)).astype(np.float32))
    wb = synth.bf16_bits_from_f32((rng.standard_normal((E * N, K)) * K ** -0.5).astype(np.float32))
    ops = (*mgw.mxfp8_quantize_rows(dev_bf16(xb), dev_i32(off)), *mgw.mxfp8_quantize_rows(dev_bf16(wb), dev_i32(w_off)))
    if not product:
        return ops, off, None
    oxq, oxs = oracle_quantize_by_expert(xb, off, oracle.token_capacity(M, E), rows=True)
    owq, ows = oracle_quantize_by_expert(wb, w_off, oracle.token_capacity(E * N, E), rows=True)
    z = np.empty((M, N))
    for _, r0, r1, v in oracle.grouped_fprop_mx_by_expert(oxq, oxs, owq, ows, off, w_off):
        z[r0:r1] = v
    return ops, off, z


def _items(counts, N):
    return sum((c + 207) // 208 for c in counts) * (N // 256)


@pytest.mark.parametrize("counts,N,K,act,bias,residual,save", [
    (MIXED, 8192, 128, "gelu", True, True, True),
    (MIXED, 8192, 896, "swiglu", True, True, True),
    ([33] * 70 + [209, 417, 300], 1024, 128, "swiglu", True, False, True),
    ([33] * 70 + [209, 417, 300], 1024, 896, "silu", False, True, False),
    ([1, 16, 17, 208] * 20, 1024, 256, "geglu", True, True, True),
])
def test_fprop_act_of_many_items_a_pair(counts, N, K, act, bias, residual, save):
    """At least four items for each pair of a 152-SM device, one after the other: both accumulators,
    their reuse, the ring and its phases across items, and epilogue warps whose first group moves on
    from item to item, also where an item has fewer groups than warps."""
    assert _items(counts, N) >= 4 * 76
    rng = np.random.default_rng(N + K)
    E, M, F = len(counts), sum(counts), N // 2 if act in GATED else N
    ops, off, z = _large_operands(rng, counts, N, K)
    b = np.float32(rng.standard_normal((E, N))) if bias else None
    res = ref.bf16(rng.standard_normal((M, F))) if residual else None
    if bias:
        z = z + np.repeat(b.astype(np.float64), counts, axis=0)
    want = ref.act(act, z) + (res if residual else 0.0)
    kw = dict(bias=None if b is None else dev(b, "f32"), residual=None if res is None else dev(res, "bf16"),
              save_preact=save)
    runs = []
    for _ in range(2):
        st = status()
        out = torch.full((M + 3, F), 77.0, dtype=torch.bfloat16, device="cuda")
        got = mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(off), M, N, ACT[act], out=out, status=st, **kw)
        assert st.item() == 0 and (out[M:] == 77).all()
        runs.append(got if save else (got, got))
    (y, zg), (y2, z2) = runs
    assert torch.equal(y, y2) and torch.equal(zg, z2)
    if save:
        assert np.all(np.abs(f64(zg) - z) <= 4e-3 * np.abs(z) + 1e-3 * np.sqrt(np.mean(z ** 2)))
    assert np.all(np.abs(f64(y[:M]) - want) <= 4e-3 * np.abs(want) + 1e-3 * np.sqrt(np.mean(want ** 2)))


@pytest.mark.parametrize("counts,N,K,act", [
    (MIXED, 8192, 128, "gelu"), (MIXED, 8192, 128, "swiglu"), ([300, 0, 129], 512, 384, "none"),
    ([40], 512, 2048, "silu"), ([16, 3], 1024, 1024, "swiglu"),    # contraction split over pairs
])
def test_the_products_residual_may_be_its_output(counts, N, K, act):
    rng = np.random.default_rng(N + K)
    M, F = sum(counts), N // 2 if act in GATED else N
    ops, off, _ = _large_operands(rng, counts, N, K, product=False)
    res = dev(rng.standard_normal((M, F)), "bf16")
    want = mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(off), M, N, ACT[act], residual=res)
    buf = res.clone()
    got = mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(off), M, N, ACT[act], residual=buf, out=buf)
    assert got is buf and torch.equal(got, want) and not torch.equal(got, res)


# ------------------------------------------------------ bias sums over long and skewed experts
@pytest.mark.parametrize("counts,N,act", [
    ([8300], 128, "none"), ([8300], 256, "swiglu"), ([0, 33000, 3], 128, "gelu"), ([0, 33000, 3], 256, "geglu"),
    ([8192 * 2, 8192], 384, "relu"),                  # eight slices
    ([2100, 0, 5000], 256, "silu"),                   # two
    ([9000] + [40] * 31, 256, "gelu"),                # one, an expert far above the mean
])
def test_bias_gradient_of_long_experts(counts, N, act):
    rng = np.random.default_rng(sum(counts) + N)
    M, F = sum(counts), N // 2 if act in GATED else N
    off = synth.offsets_from_counts(np.asarray(counts))
    dy = ref.bf16(rng.standard_normal((M, F)))
    z = ref.bf16(rng.standard_normal((M, N)))
    zt = None if act == "none" else dev(z, "bf16")
    runs = []
    for _ in range(2):
        st = status()
        dz, db = mgw.grouped_act_backward(dev(dy, "bf16"), zt, dev_i32(off), ACT[act], with_dbias=True, status=st)
        assert st.item() == 0
        runs.append((dz, db))
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
    want = ref.act_backward(act, dy, z)
    grad = np.abs(dy) if act not in GATED else \
        np.concatenate([np.abs(dy * z[:, F:]), np.abs(dy) * np.maximum(np.abs(z[:, :F]), 1)], axis=1)
    for e, n in enumerate(counts):
        rows = slice(off[e], off[e + 1])
        tol = 2.0 ** -24 * (n / 8 + 16) * np.abs(want[rows]).sum(axis=0) + 2e-6 * grad[rows].sum(axis=0)
        assert np.all(np.abs(f64(db)[e] - want[rows].sum(axis=0)) <= tol)


# ------------------------------------------------------------- dropped pairs through a layer
def _masked_layer():
    """A routing with masked experts: some tokens have fewer than top_k experts, some none."""
    T, E, K, H, N = 203, 12, 4, 256, 512
    rng = np.random.default_rng(17)
    x = np.float32(rng.standard_normal((T, E)))
    x[rng.random((T, E)) < 0.75] = -np.inf
    x[5], x[77] = -np.inf, -np.inf
    hidden = synth.bf16_bits_from_f32(rng.standard_normal((T, H)).astype(np.float32))
    wb = synth.bf16_bits_from_f32((rng.standard_normal((E * N, H)) / 16).astype(np.float32))
    return T, E, K, H, N, rng, x, hidden, wb


def test_dropped_pairs_through_a_layer():
    """The caller reads expert_off[E] back once: M, and the length of row_index that the calls take."""
    T, E, K, H, N, rng, x, hidden, wb = _masked_layer()
    st = status()
    idx, w = mgw.moe_route(dev(x, "f32"), K, status=st)
    off, row_index, row_of = mgw.moe_dispatch(idx, E, status=st)
    M = int(off[-1])
    assert 0 < M < T * K and (idx == -1).sum().item() == T * K - M
    assert (row_index[M:] == -1).all() and (row_index[:M] >= 0).all()
    row_index = row_index[:M]
    w_off = np.arange(E + 1, dtype=np.int32) * N
    xd = dev_bf16(hidden)
    xq, xs = mgw.mxfp8_quantize_rows(xd, off, row_index=row_index, status=st)
    wq, ws = mgw.mxfp8_quantize_rows(dev_bf16(wb), dev_i32(w_off), status=st)
    y, z = mgw.grouped_fprop_mxfp8_act(xq, xs, wq, ws, off, M, N, mgw.ACT_SWIGLU, save_preact=True, status=st)
    res = ref.bf16(rng.standard_normal((T, N // 2)))
    out = mgw.moe_combine(y, row_of, weights=w, residual=dev(res, "bf16"), status=st)
    # the same in 64 bits, from the router's choice on
    ri, ro, o = row_index.cpu().numpy(), row_of.cpu().numpy(), off.cpu().numpy()
    oxq, oxs = oracle.mxfp8_quantize_rows(np.ascontiguousarray(hidden[ri]), o)
    owq, ows = oracle.mxfp8_quantize_rows(wb, w_off)
    h = ref.act("swiglu", oracle.grouped_fprop_mx(oxq, oxs, owq, ows, o, w_off, M))
    rms = np.sqrt(np.mean(h ** 2))
    wf = f64(w)
    want = ref.combine(h, ro, wf, res)
    tol = ref.combine(4e-3 * np.abs(h) + 1e-3 * rms, ro, wf, None) + 2.0 ** -8 * np.abs(want) + 1e-6 * (np.abs(want) + rms)
    assert np.all(np.abs(f64(out) - want) <= tol)
    assert np.array_equal(f64(out)[[5, 77]], res[[5, 77]])      # no expert: the residual
    # and back: every gradient's call takes the same M
    dout = dev(rng.standard_normal((T, N // 2)), "bf16")
    dy, dw = mgw.moe_combine_backward(dout, y, row_of, weights=w, status=st)
    dz, db = mgw.grouped_act_backward(dy, z, off, mgw.ACT_SWIGLU, with_dbias=True, status=st)
    gq, gs = mgw.mxfp8_quantize(dz, off, status=st)
    xtq, xts = mgw.mxfp8_quantize_gather(xd, row_index, off, status=st)
    dW = mgw.grouped_wgrad_mxfp8(gq, gs, xtq, xts, off, M, status=st)
    dzq, dzs = mgw.mxfp8_quantize_rows(dz, off, status=st)
    wtq, wts = mgw.mxfp8_quantize(dev_bf16(wb), dev_i32(w_off), status=st)
    dxr = mgw.grouped_dgrad_mxfp8(dzq, dzs, wtq, wts, off, M, status=st)
    dx = mgw.moe_combine(dxr, row_of, status=st)
    dl = mgw.moe_route_backward(dev(x, "f32"), idx, dw, status=st)
    assert st.item() == 0
    for t in (dy, dz, db, dW, dx, dl):
        assert torch.isfinite(t).all()
    assert (dx[[5, 77]] == 0).all() and (dl[[5, 77]] == 0).all() and (dw[idx == -1] == 0).all()
    assert (f64(dl)[np.isinf(x)] == 0).all()
    wdz = ref.act_backward("swiglu", f64(dy), f64(z))
    assert np.all(np.abs(f64(db) - np.stack([wdz[o[e]:o[e + 1]].sum(0) for e in range(E)])) <= 1e-4)


def test_the_tables_of_all_pairs_are_refused_where_some_are_dropped():
    """Without the read: M = T * top_k is not expert_off[E], and every call says so and writes nothing."""
    T, E, K, H, N, _, x, hidden, wb = _masked_layer()
    idx, _ = mgw.moe_route(dev(x, "f32"), K)
    off, row_index, _ = mgw.moe_dispatch(idx, E)
    cap = mgw.token_capacity(T * K, E)
    st = status()
    q = torch.full((cap, H), 9, dtype=torch.uint8, device="cuda")
    mgw.mxfp8_quantize_rows(dev_bf16(hidden), off, row_index=row_index, q=q, status=st)
    assert st.item() == mgw.MGW_DEV_BAD_OFFSETS and (q == 9).all()
