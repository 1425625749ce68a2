"""The adapter operators at the limits of what a call may name: tables that are none, aliases, long sums,
every build of the kernels; against 64 bits with the tolerances of test_gpu_adapters.py."""
import ctypes

import pytest
import torch

from moe_grouped_gemm_wgrad_gb300 import build, mgw
from test_gpu_adapters import EPS, Case, own_random_numbers  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture
def clusters(monkeypatch):
    """A function that limits the clusters' size (the test build of the library takes the limit)."""
    def limit(most):
        hooks = mgw.bind(ctypes.CDLL(build.LIB_TESTHOOKS))
        monkeypatch.setattr(mgw, "load", lambda: hooks)
        monkeypatch.setenv("MGW_TEST_MAX_CLUSTER", str(most))
    return limit


def gradients_64(dy, x, u, b, off, index=None):
    """[(value, sum of absolute values)] of da and of db, on the GPU, scale 1."""
    grads = []
    rows = torch.arange(int(off[-1]), device="cuda") if index is None else index.long()
    for f in (lambda t: t.double(), lambda t: t.double().abs()):
        da, db = [], []
        for e in range(len(off) - 1):
            r = slice(int(off[e]), int(off[e + 1]))
            g, xe = f(dy[rows[r]]), f(x[rows[r]])
            da.append((g @ f(b[e])).t() @ xe)
            db.append(g.t() @ f(u[r]))
        grads.append((torch.stack(da), torch.stack(db)))
    return [(grads[0][i], grads[1][i]) for i in range(2)]


@pytest.mark.parametrize("M", [24, 500, 1400])
def test_offsets_whose_differences_wrap_are_reported(M):
    """Decreasing offsets so far apart that every 32-bit difference comes out as a positive number."""
    c = Case([M // 2, 0, M // 2], 16, 64, 128, mode="tokens")
    u = c.forward()[1]
    for table in ([0, 2 ** 31 - 1, -2, M], [0, 2 ** 30 + 7, -2 ** 30, M]):
        diffs = [(b - a + 2 ** 31) % 2 ** 32 - 2 ** 31 for a, b in zip(table, table[1:])]
        assert min(diffs) >= 0
        off = torch.tensor(table, dtype=torch.int32, device="cuda")
        outs = [torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in ((c.M, c.N), (c.M, c.K), c.a.shape, c.b.shape)]
        uu = torch.full((c.M, c.R), 7.0, device="cuda")
        mgw.grouped_lora(c.x.cuda(), c.a.cuda(), c.b.cuda(), off, out=outs[0], u=uu, **c.tables())
        assert c.status.item() == mgw.MGW_DEV_BAD_OFFSETS
        c.status.zero_()
        mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, c.a.cuda(), c.b.cuda(), off, dx=outs[1], da=outs[2],
                                  db=outs[3], **c.tables())
        assert c.status.item() == mgw.MGW_DEV_BAD_OFFSETS and (uu == 7).all() and all((t == 7).all() for t in outs)
        c.status.zero_()


@pytest.mark.parametrize("M", [30, 900, 3000])
@pytest.mark.parametrize("mode", ["tokens", "plain"])
def test_outputs_that_may_lie_on_an_input(M, mode):
    """x's own matrix (and base's at once) for out, dy's for dx without the adapters' gradients; rows in order,
    whose base and output go through one slot, and rows that lie apart."""
    c = Case([M // 2, 0, M // 3], 24, 264, 264, none=M // 6, mode=mode)
    want, u = c.forward()
    c.check_forward(want, u)
    a, b, off, tables = c.a.cuda(), c.b.cuda(), torch.from_numpy(c.off).cuda(), c.tables()
    for base in (c.base.cuda(), None, "x"):
        x = c.x.cuda()
        ex, eu = mgw.grouped_lora(x, a, b, off, base=c.x.cuda() if base == "x" else base, save_u=True, **tables)
        got, gu = mgw.grouped_lora(x, a, b, off, base=x if base == "x" else base, out=x, save_u=True, **tables)
        assert got is x and torch.equal(got, ex) and torch.equal(gu, eu)
    out = c.base.cuda()
    assert torch.equal(mgw.grouped_lora(c.x.cuda(), a, b, off, base=out, out=out, **tables), want)
    wdx = c.backward(u)[0]
    dx = c.dx_base.cuda()
    got = mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, a, b, off, dx_base=dx, dx=dx, **tables)
    assert torch.equal(got[0], wdx)
    dy = c.dy.cuda()
    got = mgw.grouped_lora_backward(dy, None, None, a, b, off, dx_base=c.dx_base.cuda(), dx=dy, with_weights=False, **tables)
    assert got[0] is dy and torch.equal(dy, wdx) and c.status.item() == 0


def test_outputs_that_may_not():
    c = Case([20, 11], 16, 64, 64, mode="plain")
    out, u = c.forward()
    a, b, off, x, dy, tables = c.a.cuda(), c.b.cuda(), torch.from_numpy(c.off).cuda(), c.x.cuda(), c.dy.cuda(), c.tables()
    twice = torch.empty(2 * c.M - 5, 64, dtype=torch.bfloat16, device="cuda")
    kept = [t.clone() for t in (x, dy, a, b, u)]
    for call in (lambda: mgw.grouped_lora_backward(dy, x, u, a, b, off, dx=dy, **tables),
                 lambda: mgw.grouped_lora_backward(dy, x, u, a, b, off, dx=x, **tables),
                 lambda: mgw.grouped_lora_backward(dy, x, u, a, b, off, da=a, **tables),
                 lambda: mgw.grouped_lora_backward(dy, x, u, a, b, off, db=b, **tables),
                 lambda: mgw.grouped_lora_backward(dy, x, u, a, b, off, dx_base=twice[:c.M], dx=twice[c.M - 5:], **tables),
                 lambda: mgw.grouped_lora(x, a, b, off, base=twice[:c.M], out=twice[c.M - 5:], **tables),
                 lambda: mgw.grouped_lora(twice[:c.M], a, b, off, out=twice[c.M - 5:], **tables)):
        with pytest.raises(mgw.MgwError, match="invalid"):
            call()
    assert all(torch.equal(p, q) for p, q in zip(kept, (x, dy, a, b, u))) and c.status.item() == 0


# A run of 256 blocks of 64 rows: 1024 additions of the tensor core, each cut off below 2^-23 of a sum no
# larger than that of the absolute values; a few, and one for every run, in fp32.
def run_error(runs):
    return (1024 + 64) * 2.0 ** -23 + runs * 2.0 ** -24


@pytest.mark.parametrize("most", [1, 8])
@pytest.mark.parametrize("M,R", [(1 << 22, 8), (1 << 20, 128)])
def test_long_sums_of_one_sign(clusters, M, R, most):
    """Sums that only grow, where additions that cut off would add up: one adapter, millions of rows."""
    clusters(most)
    g = torch.Generator(device="cuda").manual_seed(M)
    x = (torch.rand(M, 16, generator=g, device="cuda") + 1).bfloat16()
    dy = (torch.rand(M, 24, generator=g, device="cuda") + 1).bfloat16()
    u = torch.rand(M, R, generator=g, device="cuda") + 1
    a = (torch.rand(1, R, 16, generator=g, device="cuda") + 1).bfloat16()
    b = (torch.rand(1, 24, R, generator=g, device="cuda") + 1).bfloat16()
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    _, da, db = mgw.grouped_lora_backward(dy, x, u, a, b, off, with_dx=False)
    first = (24 + 64) * 2.0 ** -23
    for got, (want, size), before in zip((da, db), gradients_64(dy, x, u, b, off.tolist()), (first, 0.0)):
        err = (before + 2.0 ** -16 + run_error(M // 16384 + 1)) * size
        assert ((got.double() - want).abs() <= EPS * (want.abs() + err) + err).all()


@pytest.mark.parametrize("most", [1, 2, 3, 8])
@pytest.mark.parametrize("R", [8, 64, 72, 128])
@pytest.mark.parametrize("gathered", [False, True])
def test_adapters_around_a_run(clusters, R, most, gathered):
    """Adapters of one run and a row, of several, and of few rows, within a CTA's share and across shares."""
    clusters(most)
    counts = [16384, 5, 16385, 40001, 0, 16383, 70000, 1, 300, 33000]
    g = torch.Generator(device="cuda").manual_seed(R)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    M = off[-1]
    x = torch.randn(M, 264, generator=g, device="cuda").bfloat16()
    dy = torch.randn(M, 72, generator=g, device="cuda").bfloat16()
    a = (torch.randn(len(counts), R, 264, generator=g, device="cuda") / 16).bfloat16()
    b = (torch.randn(len(counts), 72, R, generator=g, device="cuda") / 8).bfloat16()
    perm = torch.randperm(M, generator=g, device="cuda").int() if gathered else None
    table = torch.tensor(off, dtype=torch.int32, device="cuda")
    u = torch.randn(M, R, generator=g, device="cuda")
    need = mgw.load().mgw_grouped_lora_backward_workspace_bytes(len(counts), M, 264, 72, R)
    room = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")   # nothing is read before it is written
    dx, da, db = mgw.grouped_lora_backward(dy, x, u, a, b, table, row_index=perm, out_index=perm, workspace=room[:need])
    first = (72 + 64) * 2.0 ** -23 + 2.0 ** -16
    for got, (want, size), before in zip((da, db), gradients_64(dy, x, u, b, off, perm), (first, 2.0 ** -16)):
        err = (before + run_error(5)) * size
        assert ((got.double() - want).abs() <= EPS * (want.abs() + err) + err).all()
    assert (room[need:] == 171).all()
    again = mgw.grouped_lora_backward(dy, x, u, a, b, table, row_index=perm, out_index=perm)
    assert torch.equal(again[0], dx) and torch.equal(again[1], da) and torch.equal(again[2], db)


def test_long_adapters_of_many_features():
    """More feature blocks than a cluster each leaves room for: CTAs by themselves, with sums in the workspace."""
    M, K, N, R = 16500, 16384, 4096, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    dy = torch.randn(M, N, generator=g, device="cuda").bfloat16()
    u = torch.randn(M, R, generator=g, device="cuda")
    a = (torch.randn(2, R, K, generator=g, device="cuda") / 128).bfloat16()
    b = (torch.randn(2, N, R, generator=g, device="cuda") / 8).bfloat16()
    off = torch.tensor([0, 60, M], dtype=torch.int32, device="cuda")
    need = mgw.load().mgw_grouped_lora_backward_workspace_bytes(2, M, K, N, R)
    assert need - mgw.load().mgw_grouped_lora_backward_workspace_bytes(2, 16384, K, N, R) >= 80 * 2 * 256 * R * 4
    room = torch.full((need + 4096,), 171, dtype=torch.uint8, device="cuda")
    _, da, db = mgw.grouped_lora_backward(dy, x, u, a, b, off, with_dx=False, workspace=room[:need])
    assert (room[need:] == 171).all()
    first = (N + 64) * 2.0 ** -23 + 2.0 ** -16
    cols = torch.cat([torch.arange(300), torch.arange(K - 300, K)]).cuda()   # 64-bit products are slow: some columns
    wants = gradients_64(dy[:, :256].contiguous(), x[:, :8].contiguous(), u, b[:, :256].contiguous(), [0, 60, M])
    got, (want, size) = db[:, :256], wants[1]
    err = (2.0 ** -16 + run_error(2)) * size
    assert ((got.double() - want).abs() <= EPS * (want.abs() + err) + err).all()
    for e, r in ((0, slice(0, 60)), (1, slice(60, M))):
        v, vs = dy[r].double() @ b[e].double(), dy[r].double().abs() @ b[e].double().abs()
        want, size = v.t() @ x[r][:, cols].double(), vs.t() @ x[r][:, cols].double().abs()
        err = (first + run_error(2)) * size
        assert ((da[e][:, cols].double() - want).abs() <= EPS * (want.abs() + err) + err).all()


@pytest.mark.parametrize("R", [24, 64, 128])
@pytest.mark.parametrize("mode", ["plain", "tokens", "gather"])
def test_every_build_with_more_tiles_than_sms(R, mode):
    """Two CTAs to an SM (one of rank 128, in several waves), with base and dx_base, in order and apart, in
    place too; tiles that end before, at and behind 64 rows."""
    counts = [9000, 63, 64, 65, 128 + 63, 128 + 64, 128 + 65, 0, 10100, 127, 1, 1300]
    c = Case(counts, R, 200, 456, none=77, mode=mode)
    out, u = c.forward()
    c.check_forward(out, u)
    got = c.backward(u)
    c.check_backward(u, *got)
    base, dx = c.base.cuda(), c.dx_base.cuda()
    a, b, off = c.a.cuda(), c.b.cuda(), torch.from_numpy(c.off).cuda()
    assert torch.equal(mgw.grouped_lora(c.x.cuda(), a, b, off, base=base, out=base, **c.tables()), out)
    if mode != "gather":
        again = mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, a, b, off, dx_base=dx, dx=dx, **c.tables())
        assert all(torch.equal(p, q) for p, q in zip(again, got))
    none = torch.full_like(out, 3.0)
    mgw.grouped_lora(c.x.cuda(), a, b, off, out=none, **c.tables())
    c.base = None
    c.check_forward(none, u)
    assert c.status.item() == 0


@pytest.mark.parametrize("M", [30, 900, 3000])
def test_infinities_that_meet_the_intermediate(M):
    """An infinite b (a, x, dy) beside finite intermediates: what the formula makes infinite is infinite or not a
    number (the intermediate's two parts may differ in sign, or one be 0), and all else has the same bits."""
    c = Case([M // 3, M // 3], 40, 136, 200, none=M // 3, mode="tokens")
    out, u = c.forward()
    dx, da, db = c.backward(u)
    first, second = c.o[:M // 3], c.o[M // 3:2 * (M // 3)]
    inf = float("inf")

    def same_but(got, want, hit):
        assert not got[hit].isfinite().any() and torch.equal(got[~hit], want[~hit])

    def where(t, *at):
        hit = torch.zeros_like(t, dtype=torch.bool)
        hit[at] = True
        return hit

    col = torch.arange(c.N, device="cuda")
    c.b[0, 7, 3], c.b[1, 9, 5] = inf, -inf
    got, gu = c.forward()
    hit = where(out, torch.from_numpy(first).cuda()) & (col == 7) | where(out, torch.from_numpy(second).cuda()) & (col == 9)
    same_but(got, out, hit)
    assert torch.equal(gu, u)
    c.b[0, 7, 3], c.b[1, 9, 5] = 0.5, 0.25

    out, u = c.forward()
    dx, da, db = c.backward(u)
    c.a[0, 4, 11] = inf
    got = c.backward(u)
    same_but(got[0], dx, where(dx, torch.from_numpy(first).cuda()) & (torch.arange(c.K, device="cuda") == 11))
    assert torch.equal(got[1], da) and torch.equal(got[2], db)
    c.a[0, 4, 11] = 0.5

    _, u = c.forward()
    dx, da, db = c.backward(u)
    c.x[c.t[2], 13] = -inf                     # a row of the first adapter
    got = c.backward(u)
    same_but(got[1], da, where(da, 0, slice(None), 13))
    assert torch.equal(got[0], dx) and torch.equal(got[2], db)
    c.x[c.t[2], 13] = 1.0

    dx, da, db = c.backward(u)
    c.dy[c.o[2], 21] = inf                     # its v is infinite, and with it that row of dx and all of da
    got = c.backward(u)
    same_but(got[0], dx, where(dx, int(c.o[2])))
    same_but(got[1], da, where(da, 0))
    same_but(got[2], db, where(db, 0, 21))
    assert c.status.item() == 0


@pytest.mark.parametrize("M", [30, 900, 3000])
def test_a_bad_place_of_a_row_without_an_adapter_is_reported(M):
    """Also where nothing is to be copied for it: in place, and without dx."""
    c = Case([M // 3, M // 3], 16, 64, 128, none=M // 3, mode="tokens")
    want, u = c.forward()
    bad = c.out_index.clone()
    bad[-1] = c.M
    a, b, off = c.a.cuda(), c.b.cuda(), torch.from_numpy(c.off).cuda()
    tables = dict(c.tables(), out_index=bad)
    assert c.status.item() == 0
    base, dx = c.base.cuda(), c.dx_base.cuda()
    calls = {"copied": lambda: mgw.grouped_lora(c.x.cuda(), a, b, off, base=base, **tables),
             "in place": lambda: mgw.grouped_lora(c.x.cuda(), a, b, off, base=base, out=base, **tables),
             "dx": lambda: mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, a, b, off, **tables),
             "dx in place": lambda: mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, a, b, off, dx_base=dx, dx=dx, **tables),
             "no dx": lambda: mgw.grouped_lora_backward(c.dy.cuda(), c.x.cuda(), u, a, b, off, with_dx=False, **tables)}
    for name, call in calls.items():
        call()
        assert c.status.item() == mgw.MGW_DEV_BAD_INDEX, name
        c.status.zero_()
    assert torch.equal(base[c.o[:-1]], want[c.o[:-1]])


def test_outputs_behind_the_workspace_in_one_buffer():
    """Only the bytes that the call needs of a larger workspace are its own."""
    c = Case([200, 300], 16, 64, 128, mode="tokens")
    _, u = c.forward()
    want = c.backward(u)
    need = mgw.load().mgw_grouped_lora_backward_workspace_bytes(c.E, c.M, c.K, c.N, c.R)
    arena = torch.empty(need + c.M * c.K * 2, dtype=torch.uint8, device="cuda")
    assert need % 16 == 0
    got = c.backward(u, dx=arena[need:].view(torch.bfloat16).view(c.M, c.K), workspace=arena)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    with pytest.raises(mgw.MgwError):
        c.backward(u, dx=arena[need - 16:-16].view(torch.bfloat16).view(c.M, c.K), workspace=arena)
