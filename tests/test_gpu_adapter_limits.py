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
