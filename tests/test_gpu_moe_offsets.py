"""Expert offsets that are none, so far apart that their 32-bit differences come out positive: reported by
the entry points that read offsets on their own, outputs left alone."""
import pytest
import torch

from moe_grouped_gemm_wgrad_gb300 import mgw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [300, 1200])   # one launch, and a second one for dbias
def test_act_backward(M):
    dy = torch.ones(M, 256, dtype=torch.bfloat16, device="cuda")
    dz, db = torch.full_like(dy, 5.0), torch.full((3, 256), 5.0, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for table in ([0, 2 ** 31 - 1, -2, M], [0, 2 ** 30 + 7, -2 ** 30, M]):
        assert all((b - a) % 2 ** 32 < 2 ** 31 for a, b in zip(table, table[1:]))
        off = torch.tensor(table, dtype=torch.int32, device="cuda")
        mgw.grouped_act_backward(dy, dy, off, mgw.ACT_RELU, dz=dz, dbias=db, status=st)
        assert st.item() == mgw.MGW_DEV_BAD_OFFSETS and (dz == 5).all() and (db == 5).all()
        st.zero_()
