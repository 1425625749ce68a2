"""Gradient norm and clipping on the GPU against 64 bits.

Tolerances: a thread's squares are summed in fp32 in chains of eight and a tree of eight sums (11 roundings, 2^-24
each, of a sum of positive numbers), everything after in more bits, so the sum of squares is right to
11 2^-24 and the norm, with its own rounding, to 6.5 2^-24: 2^-21.  The factor adds three roundings, an
output its own (half a step of its type); below the type's smallest normal number a step is absolute."""
import ctypes

import numpy as np
import pytest
import torch

import adapter_reference as ref
from moe_grouped_gemm_wgrad_gb300 import build, mgw

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def own_random_numbers():
    """Leaves torch's generators as it found them: other tests draw their inputs from them."""
    with torch.random.fork_rng(devices=[0]):
        torch.manual_seed(1)
        yield


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def values(rng, n, kind, size=1.0):
    return torch.from_numpy(np.float32(rng.standard_normal(n) * size)).to(TYPES[kind])


def npy(t):
    return t.double().cpu().numpy()


def check(grads, outs, norm, max_norm, eps=1e-6):
    want = ref.norm([npy(g) for g in grads])
    assert abs(norm.item() - want) <= 2.0 ** -21 * want
    f = min(1.0, max_norm / (want + eps))
    for g, o in zip(grads, outs):
        ex = npy(g) * f
        tiny = float(torch.finfo(o.dtype).tiny) * torch.finfo(o.dtype).eps
        assert o.dtype == g.dtype and o.shape == g.shape
        assert np.all(abs(npy(o) - ex) <= (2.0 ** -20 + torch.finfo(o.dtype).eps / 2) * abs(ex) + tiny)


SIZES = [[1], [7], [8], [9], [16384], [16385], [5, 0, 3, 0], [0], [100003, 1, 40000], [3] * 129, list(range(300)),
         [32768 // 2 * 3 + 5] * 3, [1] * 1500, [4096] * 1025]


@pytest.mark.parametrize("kinds", [["bf16"], ["f32"], ["bf16", "f32", "f32"]], ids="-".join)
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clip(sizes, kinds):
    rng = np.random.default_rng(len(sizes) + sum(sizes))
    host = [values(rng, n, kinds[i % len(kinds)]) for i, n in enumerate(sizes)]
    grads = [t.cuda() for t in host]
    for max_norm in (0.25, 1e9):
        outs = [torch.full_like(t, 9.0) for t in grads]
        norm = mgw.clip_grads(mgw.GradTable(grads, out=outs), max_norm)
        check(host, outs, norm, max_norm)
        assert all(torch.equal(g, h.cuda()) for g, h in zip(grads, host))
        assert torch.equal(norm, mgw.grad_norm(grads))
        # in place: the same bits
        mine = [t.clone() for t in grads]
        assert torch.equal(mgw.clip_grads(mine, max_norm), norm)
        assert all(torch.equal(p, q) for p, q in zip(mine, outs))


@pytest.mark.parametrize("sizes", [[1], [9, 0, 70001], [3] * 129], ids=lambda s: f"{len(s)}x{s[0]}")
def test_few_gradients_without_clusters(monkeypatch, sizes):
    """Where a context runs no clusters a few gradients go by the kernels for many (the test build takes the limit)."""
    rng = np.random.default_rng(sum(sizes))
    host = [values(rng, n, "bf16" if i % 2 else "f32") for i, n in enumerate(sizes)]
    grads = [t.cuda() for t in host]
    want = mgw.grad_norm(grads)
    hooks = mgw.bind(ctypes.CDLL(build.LIB_TESTHOOKS))
    monkeypatch.setattr(mgw, "load", lambda: hooks)
    for most in (1, 2, 3):
        monkeypatch.setenv("MGW_TEST_MAX_CLUSTER", str(most))
        outs = [torch.full_like(t, 9.0) for t in grads]
        norm = mgw.clip_grads(mgw.GradTable(grads, out=outs), 0.25)
        check(host, outs, norm, 0.25)
        assert (norm - want).abs().item() <= 2.0 ** -20 * want.item() and torch.equal(norm, mgw.grad_norm(grads))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_any_place_of_a_tensor(kind):
    """Views at every element offset of a 16-byte piece, lengths around a few pieces, into outputs at other
    offsets; what lies between stays as it was."""
    rng = np.random.default_rng(1)
    flat = values(rng, 9000, kind).cuda()
    at, pieces = 0, []
    for start in range(9):
        for n in (0, 1, 2, 7, 8, 9, 15, 16, 17, 40):
            at += 1 + (start * 3 + n) % 5
            pieces.append((at, n))
            at += n
    grads = [flat[p:p + n] for p, n in pieces]
    for shift in (0, 1, 3):
        dst = torch.full((at + 8,), 5.0, dtype=TYPES[kind], device="cuda")
        outs = [dst[p + shift:p + shift + n] for p, n in pieces]
        norm = mgw.clip_grads(mgw.GradTable(grads, out=outs), 2.0)
        check([g.cpu() for g in grads], outs, norm, 2.0)
        named = torch.zeros_like(dst, dtype=torch.bool)
        for p, n in pieces:
            named[p + shift:p + shift + n] = True
        assert (dst[~named] == 5).all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e-10, 1e19, 1e30, 1e36])
def test_squares_that_fp32_cannot_hold(kind, size):
    rng = np.random.default_rng(3)
    host = [values(rng, n, kind, size) for n in (40000, 3, 70001)] + [values(rng, 1000, kind, size * 1e-6)]
    grads = [t.cuda() for t in host]
    outs = [torch.empty_like(t) for t in grads]
    check(host, outs, mgw.clip_grads(mgw.GradTable(grads, out=outs), size, eps=0.0), size, eps=0.0)


def test_values_that_are_no_numbers():
    g = torch.ones(50000, device="cuda")
    g[77] = float("inf")
    out = g.clone()
    assert mgw.clip_grads([out], 1.0).item() == float("inf")
    assert torch.isnan(out[77]) and (out[:77] == 0).all() and (out[78:] == 0).all()   # inf * 0
    g[78] = float("nan")
    assert torch.isnan(mgw.clip_grads([g], 1.0)).all() and torch.isnan(g).all()
    z = torch.zeros(1000, device="cuda")
    assert mgw.clip_grads([z], 1.0).item() == 0 and not z.any()
    one = torch.ones(10, device="cuda")
    mgw.clip_grads([one], 0.0)
    assert not one.any()


def test_no_gradients_and_a_known_norm():
    assert mgw.grad_norm([]).item() == 0 and mgw.clip_grads([], 1.0).item() == 0
    g = [torch.full((1000,), 3.0, device="cuda"), torch.full((10,), 3.0, dtype=torch.bfloat16, device="cuda")]
    known = torch.tensor([30.0], device="cuda")
    assert mgw.clip_grads(g, 10.0, known_norm=known, eps=0.0) is known and known.item() == 30
    assert (g[0] == 1).all() and (g[1] == 1).all()


def test_a_tensor_past_32_bits():
    g = torch.zeros(2 ** 31 + 12345, dtype=torch.bfloat16, device="cuda")
    g[-3:], g[2 ** 31 - 2:2 ** 31 + 2] = 4.0, 2.0
    small = torch.ones(5, device="cuda")
    assert abs(mgw.grad_norm([g, small]).item() - 69 ** 0.5) <= 2.0 ** -21 * 69 ** 0.5
    mgw.clip_grads([g, small], 69 ** 0.5 / 2, eps=0.0)
    assert (g[-3:] == 2).all() and (g[2 ** 31 - 2:2 ** 31 + 2] == 1).all() and int(g.count_nonzero()) == 7


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(5)
    grads = [values(rng, n, k).cuda() for n, k in ((70000, "bf16"), (333, "f32"), (8, "bf16"))]
    outs = [torch.empty_like(t) for t in grads]
    table = mgw.GradTable(grads, out=outs)
    mgw.clip_grads(table, 1.0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = mgw.clip_grads(table, 1.0)
    for size in (3.0, 1e-4):
        for t in grads:
            t.normal_().mul_(size)
        graph.replay()
        check([t.cpu() for t in grads], outs, norm, 1.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mgw.clip_grads(table, 1.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, norm)
    # two streams at once, a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    norms = []
    for _ in range(10):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                norms.append(mgw.grad_norm(grads))
    torch.cuda.synchronize()
    assert all(torch.equal(n, norm) for n in norms)


@pytest.mark.parametrize("tokens", [50, 700])
def test_an_adapters_training_step(tokens):
    """All together as a fine-tuning step uses them: row tables, adapters beside a projection, their backward
    pass, the gradients' norm and clipping, an update, against the same step in fp64 by autograd.  Errors:
    y, dx, da and db are rounded to bf16 once (2^-8 of a value), u and what comes before them are fp32; da and
    db of a small update stay within 2^-7 of their largest value."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    E, R, K, N = 3, 16, 256, 320
    w = (torch.randn(N, K, generator=g, device="cuda") / 16).bfloat16()
    x = torch.randn(tokens, K, generator=g, device="cuda").bfloat16()
    a = (torch.randn(E, R, K, generator=g, device="cuda") / 16).bfloat16()
    b = (torch.randn(E, N, R, generator=g, device="cuda") / 4).bfloat16()
    scale = torch.tensor([0.5, 1.0, 2.0], device="cuda")
    which = torch.randint(0, E + 1, (tokens, 1), generator=g, device="cuda").int()   # E: no adapter
    dy = torch.randn(tokens, N, generator=g, device="cuda").bfloat16()

    off, rows, _ = mgw.moe_dispatch(which, E + 1)
    y = x @ w.t()
    base = y.clone()
    y, u = mgw.grouped_lora(x, a, b, off[:E + 1], row_index=rows, out_index=rows, scale=scale, base=y, out=y, save_u=True)
    dx = dy @ w
    dx_base = dx.clone()
    dx, da, db = mgw.grouped_lora_backward(dy, x, u, a, b, off[:E + 1], row_index=rows, out_index=rows, scale=scale,
                                           dx_base=dx, dx=dx)
    raw = [da.clone(), db.clone()]
    norm = mgw.clip_grads([da, db], 1.0)

    p = [t.double().requires_grad_() for t in (x, a, b)]
    delta = torch.zeros(tokens, N, dtype=torch.float64, device="cuda")
    for e in range(E):
        t = (which[:, 0] == e).nonzero().flatten()
        delta = delta.index_add(0, t, scale[e].double() * (p[0][t] @ p[1][e].t()) @ p[2][e].t())
    delta.backward(dy.double())
    for got, want in ((y, base.double() + delta.detach()), (dx, dx_base.double() + p[0].grad), (raw[0], p[1].grad),
                      (raw[1], p[2].grad)):
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-4 * want.abs().max()).all()
    want = ref.norm([npy(t) for t in raw])
    assert abs(norm.item() - want) <= 2.0 ** -21 * want and want > 1
    check([t.cpu() for t in raw], [da, db], norm, 1.0)
