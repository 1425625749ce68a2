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
from moe_grouped_gemm_wgrad_gb300 import mgw, synth
from helpers import dev_i32
from test_gpu_moe import ACT, GATED, _operands, dev, f64, status

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
