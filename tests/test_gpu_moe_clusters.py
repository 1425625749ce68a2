"""The routed-layer operators where a context cannot run the clusters that they prefer.  The test
build of the library takes a limit on the clusters' size from MGW_TEST_MAX_CLUSTER; libmgw.so asks
the device and has no such switch."""
import ctypes

import numpy as np
import pytest
import torch

import moe_reference as ref
from moe_grouped_gemm_wgrad_gb300 import build, mgw
from helpers import dev_i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def hooks():
    return mgw.bind(ctypes.CDLL(build.LIB_TESTHOOKS))


@pytest.fixture
def limited(hooks, monkeypatch):
    """Sends the binding's calls to the test build."""
    monkeypatch.setattr(mgw, "load", lambda: hooks)
    return monkeypatch


@pytest.mark.parametrize("most", [16, 8, 4, 1])
@pytest.mark.parametrize("T,K,E,drop", [
    (2049, 1, 64, 0), (683, 3, 64, 0.2), (16384, 1, 64, 0), (5462, 3, 512, 0), (8192, 8, 64, 0.05), (4097, 8, 7, 0),
    (512, 2, 513, 0), (1025, 1, 1024, 0), (8193, 1, 600, 0.1), (4096, 8, 1024, 0), (65536, 1, 1, 0),
    (100, 2, 8, 0), (8193, 8, 64, 0),     # one CTA and two launches: no clusters either way
])
def test_dispatch_with_smaller_clusters(limited, most, T, K, E, drop):
    rng = np.random.default_rng(T + K + E)
    idx = rng.integers(0, E, size=(T, K)).astype(np.int32)
    idx[rng.random((T, K)) < drop] = -1
    limited.setenv("MGW_TEST_MAX_CLUSTER", str(most))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    off, row_index, row_of = mgw.moe_dispatch(dev_i32(idx), E, status=st)
    woff, wri, wro = ref.dispatch(idx, E)
    assert st.item() == 0
    assert np.array_equal(off.cpu().numpy(), woff)
    assert np.array_equal(row_index.cpu().numpy(), wri)
    assert np.array_equal(row_of.cpu().numpy(), wro)
