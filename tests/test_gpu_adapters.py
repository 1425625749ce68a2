"""Low-rank adapters on the GPU against 64 bits (adapter_reference.py).

Tolerances, with s = sums of the products' absolute values (the same formulas on |x|, |a|, ..):
  * u: products of bf16 numbers are exact in fp32, the tensor core adds them 16 at a time and cuts off
    what lies below its accumulator's last bit (2^-23 of a sum no larger than s for each addition), the
    partial sums are added in fp32: (n + 64) 2^-23 s over a contraction of n (n / 16 additions and a
    few; far more than enough).
  * the intermediate enters the next product as two bf16 parts: 2^-8 twice, 2^-16 of its size.
  * out, dx, da, db: those errors through the second product, its own additions, and one rounding
    to bf16: 2^-8 of the value.
"""
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


EPS = 2.0 ** -8  # half a step of bf16


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def bf(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).bfloat16()


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Rows of ``counts`` adapters and ``none`` rows without one; mode 'plain': rows in order, 'tokens': a
    permutation for x and out, 'gather': x rows drawn again and again, out in row order."""

    def __init__(self, counts, R, K, N, none=0, mode="tokens", base=True, seed=0):
        rng = np.random.default_rng(sum(counts) * 31 + R + K + N + seed)
        self.E, self.R, self.K, self.N = len(counts), R, K, N
        self.off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        M = self.M = int(self.off[-1]) + none
        rows = max(1, M // 3) if mode == "gather" else M
        rows_of = {"plain": np.arange(M), "tokens": rng.permutation(M), "gather": rng.integers(0, rows, M)}[mode]
        self.t, self.o = rows_of, rows_of if mode == "tokens" else np.arange(M)
        self.row_index = None if mode == "plain" else dev(self.t.astype(np.int32))
        self.out_index = dev(self.o.astype(np.int32)) if mode == "tokens" else None
        self.x = bf(rng.standard_normal((rows, K)))
        self.a = bf(rng.standard_normal((self.E, R, K)) * K ** -0.5)
        self.b = bf(rng.standard_normal((self.E, N, R)) * R ** -0.5)
        self.scale = np.float32(rng.uniform(0.25, 2, self.E) * rng.choice([-1, 1], self.E))
        self.base = bf(rng.standard_normal((M, N))) if base else None
        self.dy = bf(rng.standard_normal((M, N)))
        self.dx_base = bf(rng.standard_normal((M, K))) if base else None
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def tables(self):
        return dict(row_index=self.row_index, out_index=self.out_index, scale=dev(self.scale), status=self.status)

    def forward(self, **kw):
        base = None if self.base is None else self.base.cuda()
        return mgw.grouped_lora(self.x.cuda(), self.a.cuda(), self.b.cuda(), dev(self.off), base=base,
                                save_u=True, **dict(self.tables(), **kw))

    def backward(self, u, **kw):
        dx_base = None if self.dx_base is None else self.dx_base.cuda()
        return mgw.grouped_lora_backward(self.dy.cuda(), self.x.cuda(), u, self.a.cuda(), self.b.cuda(), dev(self.off),
                                         dx_base=dx_base, **dict(self.tables(), **kw))

    def check_forward(self, out, u):
        x, a, b, s = f64(self.x), f64(self.a), f64(self.b), self.scale.astype(np.float64)
        base = np.zeros((self.M, self.N)) if self.base is None else f64(self.base)
        want, wu = ref.lora(x, a, b, self.off, self.t, self.o, s, base)
        su = ref.lora(abs(x), abs(a), abs(b), self.off, self.t, self.o, abs(s), 0 * base)[1]
        eu = (self.K + 64) * 2.0 ** -23 * su
        assert np.all(abs(f64(u) - wu) <= eu)
        # the second product on the intermediate's error, and on its size
        pass_on = np.zeros_like(base)
        for e in range(self.E):
            r = slice(self.off[e], self.off[e + 1])
            inner = eu[r] + (2.0 ** -16 + (2 * self.R + 64) * 2.0 ** -23) * abs(wu[r])
            pass_on[self.o[r]] = abs(s[e]) * inner @ abs(b[e]).T
        assert np.all(abs(f64(out) - want) <= EPS * (abs(want) + pass_on) + pass_on)

    def check_backward(self, u, dx, da, db):
        x, a, b, s, dy = f64(self.x), f64(self.a), f64(self.b), self.scale.astype(np.float64), f64(self.dy)
        base = np.zeros((self.M, self.K)) if self.dx_base is None else f64(self.dx_base)
        args = (f64(u), a, b, self.off, self.t, self.o, s)
        wdx, wda, wdb = ref.lora_backward(dy, x, *args, base)
        mag = [abs(v) if not isinstance(v, list) else v for v in (dy, x, f64(u), a, b)]
        sdx, sda, sdb = ref.lora_backward(*mag, self.off, self.t, self.o, abs(s), 0 * base)
        n = max(int(c) for c in np.diff(self.off)) if self.E else 0
        first = (self.N + 64) * 2.0 ** -23 + 2.0 ** -16
        for got, want, size, err in ((dx, wdx, sdx, first + (2 * self.R + 64) * 2.0 ** -23),
                                     (da, wda, sda, first + (n + 64) * 2.0 ** -23),
                                     (db, wdb, sdb, 2.0 ** -16 + (n + 64) * 2.0 ** -23)):
            err = err * size
            assert np.all(abs(f64(got) - want) <= EPS * (abs(want) + err) + err)


CASES = [
    # few rows: one row, fewer and more than a tile's eight, ranks of every width, odd sizes
    dict(counts=[1], R=8, K=8, N=8), dict(counts=[1], R=16, K=4096, N=256, mode="plain"),
    dict(counts=[0, 3, 0, 1, 0, 9, 0], R=24, K=72, N=200, none=2), dict(counts=[16], R=40, K=520, N=136, none=5),
    dict(counts=[8, 8, 7], R=64, K=264, N=1032, mode="gather", base=False), dict(counts=[20, 1], R=72, K=304, N=88),
    dict(counts=[5, 6], R=128, K=1000, N=504, none=1, mode="plain"), dict(counts=[0, 0], R=16, K=64, N=64, none=7),
    dict(counts=[250], R=104, K=96, N=64, none=6, mode="gather"), dict(counts=[1] * 200, R=8, K=32, N=40),
    # more: one tile's border, tiles of few and of many rows, no cluster and clusters
    dict(counts=[257], R=16, K=64, N=64, mode="plain"), dict(counts=[128, 129, 0, 127], R=32, K=200, N=136),
    dict(counts=[300, 3, 0, 65], R=48, K=1032, N=72, none=30, mode="gather"), dict(counts=[640], R=64, K=512, N=512, mode="plain"),
    dict(counts=[63, 64, 65, 100], R=56, K=264, N=520, mode="plain", none=1), dict(counts=[400], R=128, K=264, N=200, base=False),
    dict(counts=[200, 0, 201], R=80, K=72, N=1000, none=17), dict(counts=[17] * 40, R=8, K=2048, N=8),
    dict(counts=[700], R=24, K=8, N=328, mode="gather"), dict(counts=[0, 0, 0], R=32, K=64, N=64, none=400, mode="plain"),
    # the last rows of the kernel for few, and more than it takes, forward and backward
    dict(counts=[1024], R=32, K=64, N=72), dict(counts=[513, 511, 1], R=32, K=200, N=136, mode="plain"),
    dict(counts=[500, 12], R=40, K=96, N=64), dict(counts=[500, 0, 13], R=40, K=1032, N=520, mode="gather"),
    dict(counts=[1, 1200, 0, 127], R=8, K=520, N=264, none=9), dict(counts=[130] * 9, R=16, K=1000, N=8, base=False),
    dict(counts=[0, 1023], R=24, K=8, N=1032, none=129, mode="gather"), dict(counts=[9] * 150, R=32, K=136, N=88),
    dict(counts=[0, 0], R=16, K=64, N=328, none=1100, mode="plain"), dict(counts=[600], R=56, K=72, N=200, none=3),
    dict(counts=[500, 0, 12], R=128, K=264, N=200, base=False), dict(counts=[530, 7], R=104, K=520, N=136, none=1),
    dict(counts=[300, 0, 300], R=128, K=1000, N=264, mode="gather", base=False), dict(counts=[30] * 20, R=72, K=72, N=1000),
    # many adapters, few rows each: clusters whose CTAs have an adapter or two
    dict(counts=[1, 0, 2, 1] * 8, R=128, K=520, N=264), dict(counts=[64] * 8, R=96, K=264, N=72, mode="plain"),
    dict(counts=[0, 70, 1, 0, 130, 5], R=40, K=1000, N=328, none=40), dict(counts=[3] * 100, R=24, K=136, N=520),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(str(v) for v in c.values())[:60])
def test_forward_and_backward(case):
    c = Case(**case)
    out, u = c.forward()
    c.check_forward(out, u)
    got = c.backward(u)
    c.check_backward(u, *got)
    # the same bits again; the parts alone too
    again = c.backward(u)
    assert all(torch.equal(p, q) for p, q in zip(got, again)) and torch.equal(c.forward()[0], out)
    assert torch.equal(c.backward(None, with_weights=False)[0], got[0])
    none, da, db = c.backward(u, with_dx=False) if c.dx_base is None else (None, got[1], got[2])
    assert none is None and torch.equal(da, got[1]) and torch.equal(db, got[2])
    assert c.status.item() == 0


@pytest.mark.parametrize("M", [40, 900, 3000])
def test_in_place_and_rows_that_nobody_names(M):
    """base may be out (and dx_base dx); rows of out that no row names stay as they were."""
    c = Case([M // 2, M // 4], 16, 128, 192, none=M // 8, mode="tokens")
    want, u = c.forward()
    out = c.base.cuda()
    got, _ = mgw.grouped_lora(c.x.cuda(), c.a.cuda(), c.b.cuda(), dev(c.off), base=out, out=out, save_u=True, **c.tables())
    assert got is out and torch.equal(out, want)
    dx = c.dx_base.cuda()
    wdx = c.backward(u)[0]
    got = mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, c.a.cuda(), c.b.cuda(), dev(c.off), dx_base=dx, dx=dx, **c.tables())
    assert got[0] is dx and torch.equal(dx, wdx)
    # rows moved up by 3, into a larger out
    place = dev((c.o + 3).astype(np.int32))
    base = torch.full((c.M + 7, c.N), 2.5, dtype=torch.bfloat16, device="cuda")
    base[3:c.M + 3] = c.base.cuda()
    out = torch.full_like(base, -1.0)
    mgw.grouped_lora(c.x.cuda(), c.a.cuda(), c.b.cuda(), dev(c.off), base=base, out=out,
                     **dict(c.tables(), out_index=place))
    assert torch.equal(out[3:c.M + 3], want) and (out[:3] == -1).all() and (out[c.M + 3:] == -1).all()
    assert c.status.item() == 0


@pytest.mark.parametrize("M", [30, 600, 1800])
def test_not_a_number_stays_in_its_row_and_adapter(M):
    """Infinities and NaN in one row of x, in an unused adapter and in rows without one reach nobody else."""
    c = Case([M // 3, 0, M // 3], 16, 128, 136, none=M // 3, mode="tokens")
    x = c.x.clone()
    bad = c.t[1]
    x[bad, 5], x[bad, 6] = float("inf"), float("nan")
    x[c.t[c.off[-1]:]] = float("nan")
    a, b = c.a.clone(), c.b.clone()
    a[1], b[1] = float("nan"), float("inf")
    out, u = c.forward()
    keep = mgw.grouped_lora(x.cuda(), a.cuda(), b.cuda(), dev(c.off), base=c.base.cuda(), save_u=True, **c.tables())
    rows = np.arange(c.M) != c.o[1]
    assert torch.equal(keep[0][dev(rows)], out[dev(rows)]) and torch.isnan(keep[0][c.o[1]]).all()
    r = torch.arange(c.M, device="cuda") != 1
    assert torch.equal(keep[1][r], u[r])
    dy = c.dy.clone()
    dy[c.o[c.off[-1]:]] = float("inf")
    want = c.backward(u)
    got = mgw.grouped_lora_backward(dy.cuda(), x.cuda(), u, a.cuda(), b.cuda(), dev(c.off), dx_base=c.dx_base.cuda(), **c.tables())
    assert torch.equal(got[0], want[0])                            # dx does not read x
    assert torch.equal(got[1][1:], want[1][1:]) and torch.equal(got[2], want[2])
    assert torch.isnan(got[1][0][:, 5]).any() and torch.equal(got[1][0][:, :5], want[1][0][:, :5])


@pytest.mark.parametrize("M", [24, 500, 1400])
def test_bad_tables_are_reported(M):
    c = Case([M // 2, M // 2], 16, 64, 128, mode="tokens")
    want, u = c.forward()
    for off in ([1, M // 2, M], [0, M // 2, M + 1], [0, M // 2 + 3, M // 2], [0, -1, M]):
        out = torch.full((c.M, c.N), 7.0, dtype=torch.bfloat16, device="cuda")
        uu = torch.full((c.M, c.R), 7.0, device="cuda")
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        mgw.grouped_lora(c.x.cuda(), c.a.cuda(), c.b.cuda(), off, out=out, u=uu, **c.tables())
        assert c.status.item() == mgw.MGW_DEV_BAD_OFFSETS and (out == 7).all() and (uu == 7).all()
        c.status.zero_()
        o = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in ((c.M, c.K), c.a.shape, c.b.shape)]
        mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, c.a.cuda(), c.b.cuda(), off, dx=o[0], da=o[1], db=o[2], **c.tables())
        assert c.status.item() == mgw.MGW_DEV_BAD_OFFSETS and all((t == 7).all() for t in o)
        c.status.zero_()
    # a row of x that is none counts as zeros, a row of out that is none is not written
    rows, place = c.row_index.clone(), c.out_index.clone()
    rows[3], place[5] = c.M, -1
    base = c.base.cuda()
    out = torch.full_like(base, 7.0)
    mgw.grouped_lora(c.x.cuda(), c.a.cuda(), c.b.cuda(), dev(c.off), base=base, out=out,
                     **dict(c.tables(), row_index=rows, out_index=place))
    assert c.status.item() == mgw.MGW_DEV_BAD_INDEX
    assert torch.equal(out[c.o[3]], base[c.o[3]]) and (out[c.o[5]] == 7).all()
    rest = [r for r in range(c.M) if r not in (3, 5)]
    assert torch.equal(out[c.o[rest]], want[c.o[rest]])
    c.status.zero_()
    dx = torch.full((c.M, c.K), 7.0, dtype=torch.bfloat16, device="cuda")
    _, da, db = mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, c.a.cuda(), c.b.cuda(), dev(c.off), dx=dx,
                                          **dict(c.tables(), row_index=rows, out_index=place))
    assert c.status.item() == mgw.MGW_DEV_BAD_INDEX
    assert (dx[c.o[5]] == 7).all()
    dx[c.o[5]] = 0
    c.t, c.o, c.dx_base = c.t.copy(), c.o.copy(), None
    c.t[3], c.o[5] = -1, -1
    c.check_backward(u, dx, da, db)


def test_no_rows():
    c = Case([0, 0, 0], 16, 64, 128, mode="plain")
    out, u = c.forward()
    assert out.shape == (0, 128) and u.shape == (0, 16)
    _, da, db = c.backward(u)
    assert not da.any() and not db.any() and c.status.item() == 0


@pytest.mark.parametrize("E", [1024, 333])
def test_many_adapters(E):
    rng = np.random.default_rng(E)
    c = Case(list(rng.integers(0, 4, E) * (rng.random(E) < 0.3)), 8, 64, 72, none=3)
    out, u = c.forward()
    c.check_forward(out, u)
    c.check_backward(u, *c.backward(u))


@pytest.mark.parametrize("M", [17, 400, 1300])
def test_captured_calls_replay_on_new_data(M):
    """Two graphs, each with its own workspace, replayed in turn on inputs that change between."""
    c = Case([M // 2, M - M // 2], 32, 128, 136, mode="tokens")
    x, dy, a, b, off = c.x.cuda(), c.dy.cuda(), c.a.cuda(), c.b.cuda(), dev(c.off)
    tables = c.tables()
    graphs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            mgw.grouped_lora(x, a, b, off, save_u=True, **tables)
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, u = mgw.grouped_lora(x, a, b, off, save_u=True, **tables)
            grads = mgw.grouped_lora_backward(dy, x, u, a, b, off, **tables)
        graphs.append((g, out, u, grads))
    for step in range(4):
        x.normal_()
        dy.normal_()
        g, out, u, grads = graphs[step % 2]
        g.replay()
        eager = mgw.grouped_lora(x, a, b, off, save_u=True, **tables)
        assert torch.equal(out, eager[0]) and torch.equal(u, eager[1])
        assert all(torch.equal(p, q) for p, q in zip(grads, mgw.grouped_lora_backward(dy, x, u, a, b, off, **tables)))
    assert c.status.item() == 0


@pytest.mark.parametrize("M", [60, 700])
def test_two_streams_at_once(M):
    cases = [Case([M // 2, M // 3], 64, 512, 520, none=M // 6, seed=s) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    want = []
    for c in cases:
        out, u = c.forward()
        want.append((out, u, *c.backward(u)))
    for _ in range(8):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                out, u = c.forward()
                got.append((out, u, *c.backward(u)))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(g, w))


@pytest.mark.parametrize("most", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("case", [CASES[2], CASES[5], CASES[12], CASES[13], CASES[16], CASES[21], CASES[24], CASES[32], CASES[35], CASES[37]], ids=lambda c: str(c["counts"]))
def test_smaller_clusters(monkeypatch, most, case):
    """Where a context cannot run clusters of eight (the test build of the library takes the limit)."""
    hooks = mgw.bind(ctypes.CDLL(build.LIB_TESTHOOKS))
    monkeypatch.setattr(mgw, "load", lambda: hooks)
    monkeypatch.setenv("MGW_TEST_MAX_CLUSTER", str(most))
    c = Case(**case)
    out, u = c.forward()
    c.check_forward(out, u)
    c.check_backward(u, *c.backward(u))
    assert c.status.item() == 0


@pytest.mark.parametrize("M,E", [(20000, 3), (33000, 64)])
def test_more_tiles_than_sms(M, E):
    """Two CTAs to an SM, and tiles beyond the first wave: against a product in fp64 on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(M)
    counts = torch.bincount(torch.randint(0, E + 1, (M,), generator=g, device="cuda"), minlength=E + 1)[:E]
    off = torch.cat([torch.zeros(1, device="cuda"), counts.cumsum(0)]).int()
    perm = torch.randperm(M, generator=g, device="cuda").int()
    x = torch.randn(M, 256, generator=g, device="cuda").bfloat16()
    a = (torch.randn(E, 24, 256, generator=g, device="cuda") / 16).bfloat16()
    b = (torch.randn(E, 200, 24, generator=g, device="cuda") / 5).bfloat16()
    base = torch.randn(M, 200, generator=g, device="cuda").bfloat16()
    dy = torch.randn(M, 200, generator=g, device="cuda").bfloat16()
    out, u = mgw.grouped_lora(x, a, b, off, row_index=perm, out_index=perm, base=base, save_u=True)
    dx, da, db = mgw.grouped_lora_backward(dy, x, u, a, b, off, row_index=perm, out_index=perm)
    e = torch.searchsorted(off[1:].long(), torch.arange(M, device="cuda"), right=True)
    want, wdx = base.double(), torch.zeros(M, 256, dtype=torch.float64, device="cuda")
    for i in range(E):
        p = perm[(e == i).nonzero().flatten()].long()
        v = x[p].double() @ a[i].double().t()
        want[p] += v @ b[i].double().t()
        w = dy[p].double() @ b[i].double()
        wdx[p] = w @ a[i].double()
        for got, ex in ((da[i], w.t() @ x[p].double()), (db[i], dy[p].double().t() @ v)):
            assert ((got.double() - ex).abs() <= EPS * ex.abs() + 1e-4 * ex.abs().max()).all()
    for got, ex in ((out, want), (dx, wdx)):
        assert ((got.double() - ex).abs() <= EPS * ex.abs() + 1e-4 * ex.abs().max()).all()


def test_rows_past_32_bits():
    """x and out of more than 2^31 elements: rows at the end come out as the same rows alone."""
    M, K, N = 560000, 4096, 4096
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    x[-300:].normal_()
    g = torch.Generator(device="cuda").manual_seed(2)
    a = (torch.randn(2, 16, K, generator=g, device="cuda") / 64).bfloat16()
    b = torch.randn(2, N, 16, generator=g, device="cuda").bfloat16()
    off = torch.tensor([0, M - 170, M], dtype=torch.int32, device="cuda")
    out, u = mgw.grouped_lora(x, a, b, off, save_u=True)
    small = torch.tensor([0, 130, 300], dtype=torch.int32, device="cuda")
    want, wu = mgw.grouped_lora(x[-300:].contiguous(), a, b, small, save_u=True)
    assert not out[:-300].any()
    # Other tiles, other CTAs to a tile: another order of fp32 additions, so each side may be off by as much
    # as check_forward allows it: u by (K + 64) 2^-23 of sum |x| |a|, that and 2^-16 of |u| through b, and a
    # rounding each.
    d, ends = torch.float64, ((0, 130), (130, 300))
    for e, (lo, hi) in enumerate(ends):
        ab = b[e].to(d).abs().t()
        size = x[M - 300 + lo:M - 300 + hi].to(d).abs() @ a[e].to(d).abs().t()
        err = ((K + 64) * 2.0 ** -23 * size + (2.0 ** -16 + 96 * 2.0 ** -23) * wu[lo:hi].abs()) @ ab
        w = want[lo:hi].to(d)
        assert ((out[M - 300 + lo:M - 300 + hi].to(d) - w).abs() <= 2 * (EPS * (w.abs() + err) + err)).all()
    index = torch.arange(M - 300, M, dtype=torch.int32, device="cuda")
    got, _ = mgw.grouped_lora(x, a, b, small, row_index=index, save_u=True)
    assert torch.equal(got, want)
    got = mgw.grouped_lora_backward(want, x, wu, a, b, small, row_index=index)
    ex = mgw.grouped_lora_backward(want, x[-300:].contiguous(), wu, a, b, small)
    assert all(torch.equal(p, q) for p, q in zip(got, ex))


@pytest.mark.parametrize("M", [16, 700, 5000])
def test_inputs_written_just_before_and_read_just_after(M):
    """Launches that begin while the one before ends: inputs written, outputs overwritten and read by the
    launches next to a call's, eagerly, captured, and captured behind a join of two streams."""
    c = Case([M // 2, M // 3], 32, 512, 520, none=M // 6, mode="tokens")
    a, b, off, tables = c.a.cuda(), c.b.cuda(), dev(c.off), c.tables()
    xs = [torch.randn(M // 2 + M // 3 + M // 6, 512, device="cuda").bfloat16() for _ in range(4)]
    dys = [torch.randn(len(xs[0]), 520, device="cuda").bfloat16() for _ in range(4)]
    want = []
    for x, dy in zip(xs, dys):
        out, u = mgw.grouped_lora(x, a, b, off, save_u=True, **tables)
        torch.cuda.synchronize()
        grads = mgw.grouped_lora_backward(dy, x, u, a, b, off, **tables)
        norm = mgw.clip_grads(list(grads), 0.5)
        torch.cuda.synchronize()
        want.append((out, u, *grads, norm))
    x, dy, noise = torch.empty_like(xs[0]), torch.empty_like(dys[0]), torch.randn(1 << 22, device="cuda")
    out, u = torch.empty_like(want[0][0]), torch.empty_like(want[0][1])

    def step(x_now, dy_now, side=None):
        if side is not None:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                noise.mul_(1.0)
                dy.copy_(dy_now)
        else:
            dy.copy_(dy_now)
        out.fill_(9.0)
        x.copy_(x_now)
        if side is not None:
            torch.cuda.current_stream().wait_stream(side)
        mgw.grouped_lora(x, a, b, off, out=out, u=u, **tables)
        kept = [out.clone(), u.clone()]
        out.fill_(7.0)
        grads = mgw.grouped_lora_backward(dy, x, u, a, b, off, **tables)
        u.zero_()
        norm = mgw.clip_grads(list(grads), 0.5)
        result = (*kept, *[t.clone() for t in grads], norm.clone())
        for t in grads:
            t.zero_()
        return result

    def same(got, ex):
        return all(torch.equal(p, q) for p, q in zip(got, ex))

    side = torch.cuda.Stream()
    got = [step(xs[i % 4], dys[i % 4], side if i % 3 == 0 else None) for i in range(24)]
    torch.cuda.synchronize()
    assert all(same(g, want[i % 4]) for i, g in enumerate(got))
    in_x, in_dy = xs[0].clone(), dys[0].clone()
    for fork in (None, side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step(in_x, in_dy, fork)
        for i in range(8):
            in_x.copy_(xs[i % 4])
            in_dy.copy_(dys[i % 4])
            graph.replay()
            assert same(got, want[i % 4])
    # a call as a graph's first node, alone, and two calls in a row
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = mgw.grouped_lora(in_x, a, b, off, save_u=True, **tables)
        second = mgw.grouped_lora_backward(in_dy, in_x, first[1], a, b, off, **tables)
    for i in range(4):
        in_x.copy_(xs[i % 4])
        in_dy.copy_(dys[i % 4])
        graph.replay()
        norm = mgw.clip_grads(list(second), 0.5)
        assert same((*first, *second, norm), want[i % 4])
    assert c.status.item() == 0
