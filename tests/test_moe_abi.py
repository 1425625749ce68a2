"""The routed-layer entry points on the host: argument errors return codes before any device
work, and the binding refuses what the tensors show to be wrong (with a stand-in library)."""
import contextlib
import ctypes

import pytest
import torch

from moe_grouped_gemm_wgrad_gb300 import build, mgw

P = ctypes.c_void_p
OK = P(0x1000)     # never dereferenced: validation fails first
ODD = P(0x1008)    # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mgw.load()


def _call(fn, base, **changes):
    a = dict(base, **changes)
    return fn(*a.values())


def test_route_refusals(lib):
    base = dict(logits=OK, dtype=0, T=4, E=64, bias=None, top_k=8, score=0, groups=1, top_groups=1,
                group_best=1, renorm=1, scale=1.0, idx=OK, w=OK, scores=None, status=None, stream=None)
    for bad in (dict(logits=None), dict(idx=None), dict(w=None), dict(dtype=2), dict(T=-1), dict(E=0),
                dict(E=1025), dict(top_k=0), dict(top_k=33), dict(E=4), dict(score=2), dict(groups=0),
                dict(groups=33), dict(groups=4, top_groups=5), dict(top_groups=0), dict(group_best=3),
                dict(logits=ODD), dict(bias=ODD), dict(idx=ODD), dict(w=ODD), dict(scores=ODD)):
        assert _call(lib.mgw_moe_route, base, **bad) == -1, bad
    assert _call(lib.mgw_moe_route, base, E=66, groups=4, top_groups=2) == -2


def test_route_backward_refusals(lib):
    base = dict(logits=OK, dtype=0, T=4, E=64, top_k=8, score=0, renorm=1, scale=1.0, idx=OK, dw=OK,
                ds=None, dl=OK, status=None, stream=None)
    for bad in (dict(logits=None), dict(idx=None), dict(dl=None), dict(dtype=-1), dict(T=-1),
                dict(E=0), dict(top_k=0), dict(top_k=65), dict(score=-1), dict(dw=ODD), dict(ds=ODD),
                dict(dl=ODD), dict(logits=ODD), dict(idx=ODD)):
        assert _call(lib.mgw_moe_route_backward, base, **bad) == -1, bad


def test_dispatch_refusals(lib):
    base = dict(idx=OK, T=4, top_k=2, E=8, off=OK, ri=OK, ro=OK, ws=None, n=0, status=None, stream=None)
    for bad in (dict(idx=None), dict(off=None), dict(ri=None), dict(ro=None), dict(T=-1),
                dict(top_k=0), dict(top_k=33), dict(E=0), dict(E=1025), dict(idx=ODD), dict(off=ODD),
                dict(ri=ODD), dict(ro=ODD), dict(ws=ODD), dict(T=1 << 20)):
        assert _call(lib.mgw_moe_dispatch, base, **bad) == -1, bad
    assert _call(lib.mgw_moe_dispatch, base, T=1 << 29, top_k=4, ws=OK, n=1 << 30) == -2
    need = lib.mgw_moe_dispatch_workspace_bytes(1 << 20, 2, 8)
    assert need > 0 and need % 32 == 0
    assert _call(lib.mgw_moe_dispatch, base, T=1 << 20, ws=OK, n=need - 1) == -3
    assert lib.mgw_moe_dispatch_workspace_bytes(4, 2, 8) == 0
    assert lib.mgw_moe_dispatch_workspace_bytes(-1, 2, 8) == 0


def test_fprop_act_refusals(lib):
    base = dict(xq=OK, xs=OK, wq=OK, ws=OK, off=OK, E=1, M=4, N=256, K=128, Mcap=256, Mw=256, act=2,
                bias=None, res=None, y=OK, z=None, status=None, stream=None)
    fn = lib.mgw_grouped_fprop_mxfp8_act
    for bad in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(off=None), dict(y=None),
                dict(M=-1), dict(N=0), dict(K=0), dict(E=0), dict(E=1025), dict(act=-1), dict(act=6),
                dict(xq=ODD), dict(xs=ODD), dict(wq=ODD), dict(ws=ODD), dict(bias=ODD), dict(res=ODD),
                dict(y=ODD), dict(z=ODD)):
        assert _call(fn, base, **bad) == -1, bad
    for bad in (dict(N=128), dict(K=64), dict(N=384)):
        assert _call(fn, base, **bad) == -2, bad
    for bad in (dict(Mcap=128), dict(Mcap=250), dict(Mw=128), dict(Mw=300)):
        assert _call(fn, base, **bad) == -3, bad


def test_act_backward_refusals(lib):
    base = dict(dy=OK, z=OK, off=OK, E=2, M=3000, N=256, act=2, dz=OK, db=None, ws=None, n=0, status=None,
                stream=None)
    fn = lib.mgw_grouped_act_backward
    for bad in (dict(dy=None), dict(z=None), dict(off=None), dict(dz=None), dict(E=0), dict(E=1025),
                dict(M=-1), dict(N=0), dict(act=-1), dict(act=6), dict(db=OK), dict(dy=ODD), dict(z=ODD),
                dict(dz=ODD), dict(db=ODD, ws=OK, n=1 << 30), dict(ws=ODD)):
        assert _call(fn, base, **bad) == -1, bad
    assert _call(fn, base, N=192) == -2
    assert _call(fn, base, N=128, act=4) == -2
    need = lib.mgw_grouped_act_backward_workspace_bytes(2, 3000, 256)
    assert need >= (23 + 2) * 256 * 4   # a row of sums per row tile of either expert
    assert _call(fn, base, db=OK, ws=OK, n=need - 1) == -3
    assert lib.mgw_grouped_act_backward_workspace_bytes(0, 3000, 256) == 0


def test_combine_refusals(lib):
    base = dict(y=OK, dtype=0, M=8, ro=OK, w=OK, res=None, T=4, top_k=2, H=64, out=OK, status=None,
                stream=None)
    for bad in (dict(y=None), dict(ro=None), dict(out=None), dict(dtype=5), dict(M=-1), dict(T=-1),
                dict(top_k=0), dict(top_k=33), dict(H=0), dict(y=ODD), dict(ro=ODD), dict(w=ODD),
                dict(res=ODD), dict(out=ODD)):
        assert _call(lib.mgw_moe_combine, base, **bad) == -1, bad
    assert _call(lib.mgw_moe_combine, base, H=(1 << 23) + 1) == -2
    base = dict(dout=OK, y=OK, dtype=1, M=8, ro=OK, w=OK, T=4, top_k=2, H=64, dy=OK, dw=OK, status=None,
                stream=None)
    for bad in (dict(dout=None), dict(y=None), dict(ro=None), dict(dy=None), dict(dtype=5),
                dict(dout=ODD), dict(y=ODD), dict(ro=ODD), dict(w=ODD), dict(dy=ODD), dict(dw=ODD)):
        assert _call(lib.mgw_moe_combine_backward, base, **bad) == -1, bad


# ------------------------------------------------------------------ the binding's checks
class StandIn:
    def __init__(self):
        self.calls = []

    def mgw_mxfp8_scale_bytes(self, C, Mcap):
        return C * Mcap // 32

    def mgw_moe_dispatch_workspace_bytes(self, T, K, E):
        return 64 if T > 100 else 0

    def mgw_grouped_act_backward_workspace_bytes(self, E, M, N):
        return 4 * (M // 128 + E) * N

    def __getattr__(self, name):
        if not name.startswith("mgw_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append(name)
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    f = StandIn()
    monkeypatch.setattr(mgw, "load", lambda: f)
    monkeypatch.setattr(mgw, "_on_cuda", lambda t: True)
    monkeypatch.setattr(mgw, "_device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(mgw, "_stream", lambda s: None)
    return f


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(s, dtype=torch.float32)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def _rejects(fake, fn, *args, **kw):
    with pytest.raises(mgw.MgwError):
        fn(*args, **kw)
    assert fake.calls == []


def test_binding_route(fake):
    idx, w = mgw.moe_route(bf(4, 16), 2)
    assert idx.shape == w.shape == (4, 2) and fake.calls == ["mgw_moe_route"]
    assert len(mgw.moe_route(f32(4, 16), 2, with_scores=True)) == 3
    assert mgw.moe_route_backward(f32(4, 16), idx, w, dscores=f32(4, 16)).dtype == torch.float32
    fake.calls.clear()
    for bad in (lambda: (bf(4, 16).half(), 2), lambda: (bf(16), 2), lambda: (bf(16, 4).t(), 2),
                lambda: (bf(4, 16), 0), lambda: (bf(4, 16), 17)):
        _rejects(fake, mgw.moe_route, *bad())
    _rejects(fake, mgw.moe_route, bf(4, 16), 2, bias=bf(16))
    _rejects(fake, mgw.moe_route, bf(4, 16), 2, bias=f32(15))
    _rejects(fake, mgw.moe_route, bf(4, 16), 2, weights=f32(4, 1))
    _rejects(fake, mgw.moe_route, bf(4, 16), 2, scores=f32(4, 15))
    _rejects(fake, mgw.moe_route, bf(4, 16), 2, expert_idx=f32(4, 2))
    _rejects(fake, mgw.moe_route_backward, bf(4, 16), i32(3, 2), f32(3, 2))
    _rejects(fake, mgw.moe_route_backward, bf(4, 16), i32(4, 2), f32(4, 3))
    _rejects(fake, mgw.moe_route_backward, bf(4, 16), i32(4, 2), None, dscores=f32(4, 15))
    _rejects(fake, mgw.moe_route_backward, bf(4, 16), i32(4, 2), f32(4, 2), dlogits=f32(4, 16))


def test_binding_dispatch(fake):
    off, ri, ro = mgw.moe_dispatch(i32(5, 2), 3)
    assert off.shape == (4,) and ri.shape == (10,) and ro.shape == (5, 2)
    assert fake.calls == ["mgw_moe_dispatch"]
    fake.calls.clear()
    _rejects(fake, mgw.moe_dispatch, i32(10), 3)
    _rejects(fake, mgw.moe_dispatch, i32(5, 2).long(), 3)
    _rejects(fake, mgw.moe_dispatch, i32(5, 2), 0)
    _rejects(fake, mgw.moe_dispatch, i32(5, 2), 3, expert_off=i32(3))
    _rejects(fake, mgw.moe_dispatch, i32(5, 2), 3, row_index=i32(9))
    _rejects(fake, mgw.moe_dispatch, i32(500, 2), 3, workspace=u8(63))


def test_binding_product(fake):
    off = torch.tensor([0, 10, 20], dtype=torch.int32)
    ops = (u8(384, 128), u8(384 * 4), u8(512, 128), u8(512 * 4), off)
    y = mgw.grouped_fprop_mxfp8_act(*ops, 20, 256, mgw.ACT_SWIGLU)
    assert y.shape == (20, 128)
    y, z = mgw.grouped_fprop_mxfp8_act(*ops, 20, 256, mgw.ACT_GELU, save_preact=True)
    assert y.shape == z.shape == (20, 256)
    dz, db = mgw.grouped_act_backward(bf(20, 128), z, off, mgw.ACT_GEGLU, with_dbias=True)
    assert dz.shape == (20, 256) and db.shape == (2, 256)
    dy = bf(20, 256)
    assert mgw.grouped_act_backward(dy, None, off, mgw.ACT_NONE, with_dbias=True)[0] is dy
    fake.calls.clear()
    _rejects(fake, mgw.grouped_fprop_mxfp8_act, *ops, 20, 256, mgw.ACT_GELU, bias=f32(2, 255))
    _rejects(fake, mgw.grouped_fprop_mxfp8_act, *ops, 20, 256, mgw.ACT_GELU, bias=bf(2, 256))
    _rejects(fake, mgw.grouped_fprop_mxfp8_act, *ops, 20, 256, mgw.ACT_SWIGLU, residual=bf(20, 256))
    _rejects(fake, mgw.grouped_fprop_mxfp8_act, *ops, 20, 256, mgw.ACT_NONE, out=bf(19, 256))
    _rejects(fake, mgw.grouped_fprop_mxfp8_act, *ops, 20, 256, mgw.ACT_SWIGLU, preact=bf(20, 128))
    _rejects(fake, mgw.grouped_fprop_mxfp8_act, u8(384, 128), u8(10), *ops[2:], 20, 256)
    _rejects(fake, mgw.grouped_act_backward, bf(20, 256), None, off, mgw.ACT_RELU)
    _rejects(fake, mgw.grouped_act_backward, bf(20, 256), bf(20, 256), off, mgw.ACT_SWIGLU)
    _rejects(fake, mgw.grouped_act_backward, bf(20, 256), bf(20, 256), off, mgw.ACT_NONE)
    _rejects(fake, mgw.grouped_act_backward, bf(20, 256), bf(20, 256), off, mgw.ACT_RELU, dbias=f32(2, 255))
    _rejects(fake, mgw.grouped_act_backward, bf(20, 256), bf(20, 256), off, mgw.ACT_RELU, with_dbias=True,
             workspace=u8(1))


def test_binding_combine(fake):
    y, ro, w = bf(10, 64), i32(5, 2), f32(5, 2)
    assert mgw.moe_combine(y, ro, weights=w, residual=bf(5, 64)).shape == (5, 64)
    dy, dw = mgw.moe_combine_backward(bf(5, 64), y, ro, weights=w)
    assert dy.shape == (10, 64) and dw.shape == (5, 2)
    assert mgw.moe_combine_backward(bf(5, 64), None, ro, M=10)[1] is None
    fake.calls.clear()
    _rejects(fake, mgw.moe_combine, y.half(), ro)
    _rejects(fake, mgw.moe_combine, y, ro.long())
    _rejects(fake, mgw.moe_combine, y, ro, weights=f32(5, 3))
    _rejects(fake, mgw.moe_combine, y, ro, residual=f32(5, 64))
    _rejects(fake, mgw.moe_combine, y, ro, out=bf(4, 64))
    _rejects(fake, mgw.moe_combine_backward, bf(5, 64), None, ro, weights=w)
    _rejects(fake, mgw.moe_combine_backward, bf(5, 64), None, ro)
    _rejects(fake, mgw.moe_combine_backward, bf(5, 64), f32(10, 64), ro, weights=w)
    _rejects(fake, mgw.moe_combine_backward, bf(5, 64), y, ro, M=11, weights=w)
    _rejects(fake, mgw.moe_combine_backward, bf(5, 64), y, ro, dweights=w)


def test_cluster_limit_only_in_the_test_build():
    build.build()
    with open(build.LIB, "rb") as f:
        assert b"MGW_TEST_MAX_CLUSTER" not in f.read()
    with open(build.LIB_TESTHOOKS, "rb") as f:
        assert b"MGW_TEST_MAX_CLUSTER" in f.read()
