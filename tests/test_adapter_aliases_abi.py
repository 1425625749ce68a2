"""Outputs of the adapter entry points that overlap each other or an input are refused before any device work."""
import ctypes
import itertools

import pytest

from moe_grouped_gemm_wgrad_gb300 import build, mgw

P = ctypes.c_void_p
GAP = 1 << 26         # addresses are never dereferenced
E, R, K, N, M, ROWS = 2, 16, 64, 48, 8, 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mgw.load()


def _sizes(**s):
    """name -> (address, bytes), far from each other."""
    return {k: (GAP * (i + 1), n) for i, (k, n) in enumerate(s.items())}


def _forward(lib, at, k=K):
    p = {n: None if v is None else P(v) for n, v in at.items()}
    return lib.mgw_grouped_lora(p["x"], ROWS, p["row"], M, k, p["a"], p["b"], p["scale"], p["off"], E, R, N, p["base"],
                                p["place"], ROWS, p["out"], p["u"], None, None)


def _backward(lib, at, need, k=K):
    p = {n: None if v is None else P(v) for n, v in at.items()}
    return lib.mgw_grouped_lora_backward(p["dy"], ROWS, p["place"], p["x"], ROWS, p["row"], M, k, p["a"], p["b"],
                                         p["scale"], p["off"], E, R, N, p["u"], p["base"], p["dx"], p["da"], p["db"],
                                         p["ws"], need, None, None)


def _places(spans, out, other):
    """Addresses of ``out`` that overlap ``other``: on it, its last 16 bytes, and from before into it."""
    start, n = spans[other]
    size = spans[out][1]
    return {start, start + (n - 1) // 16 * 16, start - (size - 1) // 16 * 16}


INPUTS = dict(a=E * R * K * 2, b=E * N * R * 2, scale=E * 4, off=(E + 1) * 4, row=M * 4, place=M * 4)


def test_forward(lib):
    spans = _sizes(x=ROWS * K * 2, base=ROWS * N * 2, out=ROWS * N * 2, u=M * R * 4, **INPUTS)
    at = {k: v[0] for k, v in spans.items()}
    for out, other in itertools.product(("out", "u"), spans):
        if out == other:
            continue
        for place in _places(spans, out, other):
            if (out, other, place) != ("out", "base", spans["base"][0]):   # base may be out
                assert _forward(lib, dict(at, **{out: place})) == -1, (out, other, place)


def test_backward(lib):
    need = lib.mgw_grouped_lora_backward_workspace_bytes(E, M, K, N, R)
    assert 0 < need
    spans = _sizes(dy=ROWS * N * 2, x=ROWS * K * 2, base=ROWS * K * 2, u=M * R * 4, dx=ROWS * K * 2, da=E * R * K * 2,
                   db=E * N * R * 2, **INPUTS, ws=need)
    at = {k: v[0] for k, v in spans.items()}
    for out, other in itertools.product(("dx", "da", "db", "ws"), spans):
        if out == other:
            continue
        for place in _places(spans, out, other):
            if (out, other, place) != ("dx", "base", spans["base"][0]):    # dx_base may be dx
                assert _backward(lib, dict(at, **{out: place}), need) == -1, (out, other, place)


def test_the_other_directions_matrix_of_the_same_width(lib):
    """dx on dy where dy is read again for dB; without that, only dy's own place."""
    need = lib.mgw_grouped_lora_backward_workspace_bytes(E, M, N, N, R)
    spans = _sizes(dy=ROWS * N * 2, x=ROWS * N * 2, base=ROWS * N * 2, u=M * R * 4, dx=ROWS * N * 2, da=E * R * N * 2,
                   db=E * N * R * 2, **INPUTS, ws=need)
    at = dict({k: v[0] for k, v in spans.items()}, base=None)
    assert _backward(lib, dict(at, dx=at["dy"]), need, k=N) == -1
    alone = dict(at, da=None, db=None, ws=None)
    assert _backward(lib, dict(alone, dx=at["dy"] + N * 2), 0, k=N) == -1
    assert _backward(lib, dict(alone, dx=at["dy"]), 0, k=N - 8) == -1
    assert _forward(lib, dict(at, base=None, out=at["x"] + 96), k=N) == -1
