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
from test_gpu_moe import ACT, GATED, _operands, dev, f64

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


@pytest.mark.parametrize("most", [8, 4, 2])
@pytest.mark.parametrize("counts,N,K,act", [([16], 1024, 2048, "swiglu"), ([0, 33, 0, 31], 256, 1024, "gelu"),
                                            ([5, 7], 512, 640, "none"), ([1], 256, 512, "silu")])
def test_product_with_smaller_clusters(limited, most, counts, N, K, act):
    """Contractions split over clusters of four pairs, of two, and not at all: the tolerance is that of
    test_fprop_act."""
    rng = np.random.default_rng(sum(counts) + N + K)
    ops, off, z = _operands(rng, counts, N, K)
    M, F = sum(counts), N // 2 if act in GATED else N
    b = np.float32(rng.standard_normal((len(counts), N)))
    want = ref.act(act, z + np.repeat(b.astype(np.float64), counts, axis=0))
    limited.setenv("MGW_TEST_MAX_CLUSTER", str(most))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = mgw.grouped_fprop_mxfp8_act(*ops, dev_i32(off), M, N, ACT[act], bias=dev(b, "f32"), status=st)
    assert st.item() == 0 and got.shape == (M, F)
    assert np.all(np.abs(f64(got) - want) <= 4e-3 * np.abs(want) + 1e-3 * np.sqrt(np.mean(want ** 2)))
