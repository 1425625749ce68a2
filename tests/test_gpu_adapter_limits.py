"""The adapter operators at the limits of what a call may name: tables that are none, aliases, long sums,
every build of the kernels; against 64 bits with the tolerances of test_gpu_adapters.py."""
import pytest
import torch

from moe_grouped_gemm_wgrad_gb300 import mgw
from test_gpu_adapters import Case, own_random_numbers  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


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
