"""The adapter and gradient entry points on the host: argument errors return codes before any device
work; the binding refuses what the tensors show to be wrong, and runs on the stream it is given (with
a stand-in library)."""
import contextlib
import ctypes

import pytest
import torch

from moe_grouped_gemm_wgrad_gb300 import adapters, build, gradients, mgw

P = ctypes.c_void_p
OK = P(0x1000)     # never dereferenced: validation fails first
ODD = P(0x1008)    # not 16-byte aligned


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mgw.load()


def _call(fn, args, /, **changes):
    return fn(*dict(args, **changes).values())


def test_lora_refusals(lib):
    base = dict(x=OK, x_rows=8, ri=None, M=8, K=64, a=OK, b=OK, scale=None, off=OK, E=2, R=16, N=64, base=None,
                oi=None, out_rows=8, out=OK, u=None, status=None, stream=None)
    for bad in (dict(x=None), dict(a=None), dict(b=None), dict(off=None), dict(out=None), dict(M=-1), dict(K=0),
                dict(N=-8), dict(R=0), dict(E=0), dict(E=1025), dict(x_rows=7), dict(out_rows=7), dict(x_rows=-1),
                dict(ri=OK, x_rows=0), dict(oi=OK, out_rows=0), dict(x=ODD), dict(ri=ODD), dict(a=ODD), dict(b=ODD),
                dict(scale=ODD), dict(off=ODD), dict(base=ODD), dict(oi=ODD), dict(out=ODD), dict(u=ODD)):
        assert _call(lib.mgw_grouped_lora, base, **bad) == -1, bad
    for bad in (dict(K=60), dict(N=4), dict(R=12), dict(R=136), dict(K=(1 << 23) + 8), dict(N=(1 << 23) + 8),
                dict(M=(1 << 30) + 1, x_rows=2 ** 31 - 1, out_rows=2 ** 31 - 1)):
        assert _call(lib.mgw_grouped_lora, base, **bad) == -2, bad


def test_lora_backward_refusals(lib):
    need = lib.mgw_grouped_lora_backward_workspace_bytes(2, 8, 64, 64, 16)
    base = dict(dy=OK, out_rows=8, oi=None, x=OK, x_rows=8, ri=None, M=8, K=64, a=OK, b=OK, scale=None, off=OK, E=2,
                R=16, N=64, u=OK, dx_base=None, dx=OK, da=OK, db=OK, ws=OK, n=need, status=None, stream=None)
    fn = lib.mgw_grouped_lora_backward
    for bad in (dict(dy=None), dict(x=None), dict(u=None), dict(a=None), dict(b=None), dict(off=None), dict(da=None),
                dict(db=None), dict(ws=None), dict(dx=None, dx_base=OK), dict(M=9), dict(M=-1), dict(E=0), dict(R=0),
                dict(dy=ODD), dict(x=ODD), dict(u=ODD), dict(dx=ODD), dict(da=ODD), dict(db=ODD), dict(ws=ODD),
                dict(dx_base=ODD), dict(oi=ODD), dict(ri=ODD)):
        assert _call(fn, base, **bad) == -1, bad
    for bad in (dict(K=60), dict(N=4), dict(R=12), dict(R=136)):
        assert _call(fn, base, **bad) == -2, bad
    assert _call(fn, base, n=need - 1) == -3
    size = lib.mgw_grouped_lora_backward_workspace_bytes
    assert size(2, 8, 64, 64, 16) > 0 and size(1, 0, 64, 64, 16) >= 0
    assert size(0, 8, 64, 64, 16) == size(2, -1, 64, 64, 16) == size(2, 8, 64, 64, 129) == 0
    # two blocks of 64 rows for each row tile, high and low parts, of u and of v
    assert size(4, 1000, 8192 * 8, 8192 * 8, 16) == 2 * (1000 // 128 + 4) * 2 * 256 * 16


def _arrays(ptrs, sizes, kinds):
    n = len(ptrs)
    return (P * n)(*ptrs), (ctypes.c_int64 * n)(*sizes), (ctypes.c_int * n)(*kinds)


def test_grad_refusals(lib):
    need = lib.mgw_grad_workspace_bytes(2)
    assert need > 0 and lib.mgw_grad_workspace_bytes(-1) == 0 and lib.mgw_grad_workspace_bytes(3000) == 3 * need
    g, s, k = _arrays([0x1000, 0x2002], [5, 7], [1, 0])
    norm = dict(g=g, s=s, k=k, n=2, norm=OK, ws=OK, size=need, stream=None)
    clip = dict(g=g, o=None, s=s, k=k, n=2, max_norm=1.0, eps=1e-6, norm_in=None, norm=OK, ws=OK, size=need, stream=None)
    bad_ptr, bad_size, bad_kind = _arrays([0x1002, 0x2002], [5, -1], [2, 0])   # an fp32 number at an odd place
    null = _arrays([0, 0x2002], [5, 7], [1, 0])[0]
    huge = _arrays([0, 0], [1 << 41, 0], [0, 0])[1]
    for fn, base in ((lib.mgw_grad_norm, norm), (lib.mgw_grad_clip, clip)):
        for bad in (dict(g=None), dict(s=None), dict(k=None), dict(n=-1), dict(g=bad_ptr), dict(g=null),
                    dict(s=bad_size), dict(k=bad_kind), dict(norm=None), dict(norm=P(0x1002)), dict(ws=None), dict(ws=ODD)):
            assert _call(fn, base, **bad) == -1, bad
        assert _call(fn, base, s=huge) == -2
        assert _call(fn, base, size=need - 1) == -3
    for bad in (dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1e-6), dict(eps=float("nan")),
                dict(norm_in=OK), dict(norm=None), dict(o=bad_ptr), dict(o=null)):
        assert _call(lib.mgw_grad_clip, clip, **bad) == -1, bad


# ---------------------------------------------------------------------------------- the binding
class FakeLib:
    def __init__(self):
        self.calls = []

    def mgw_grouped_lora_backward_workspace_bytes(self, *sizes):
        return 64

    def mgw_grad_workspace_bytes(self, n):
        return 64

    def mgw_status_string(self, st):
        return b"stand-in"

    def __getattr__(self, name):
        if not name.startswith("mgw_"):
            raise AttributeError(name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    f = FakeLib()
    monkeypatch.setattr(mgw, "load", lambda: f)
    monkeypatch.setattr(mgw, "_on_cuda", lambda t: True)
    monkeypatch.setattr(mgw, "_device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(mgw, "_stream", lambda s: None)
    return f


def bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def f32(*s):
    return torch.zeros(s)


def i32(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_reached_through_mgw():
    assert mgw.grouped_lora is adapters.grouped_lora and mgw.clip_grads is gradients.clip_grads
    assert mgw.GradTable is gradients.GradTable
    with pytest.raises(AttributeError):
        mgw.no_such_operator


X, A, B, OFF = (10, 64), (3, 16, 64), (3, 48, 16), 4   # rows, adapters of rank 16, 64 -> 48 columns


def test_lora_shapes(fake):
    out = mgw.grouped_lora(bf(*X), bf(*A), bf(*B), i32(OFF))
    assert out.shape == (10, 48) and fake.calls[-1][0] == "mgw_grouped_lora" and fake.calls[-1][1][3] == 10
    out, u = mgw.grouped_lora(bf(*X), bf(*A), bf(*B), i32(OFF), row_index=i32(25), base=bf(25, 48), save_u=True)
    assert out.shape == (25, 48) and u.shape == (25, 16)
    assert mgw.grouped_lora(bf(*X), bf(*A), bf(*B), i32(OFF), row_index=i32(4), out_index=i32(4), base=bf(9, 48)).shape == (9, 48)
    base = bf(10, 48)
    assert mgw.grouped_lora(bf(*X), bf(*A), bf(*B), i32(OFF), base=base, out=base) is base
    dx, da, db = mgw.grouped_lora_backward(bf(10, 48), bf(*X), f32(10, 16), bf(*A), bf(*B), i32(OFF))
    assert dx.shape == (10, 64) and da.shape == A and db.shape == B
    dx, da, db = mgw.grouped_lora_backward(bf(10, 48), None, None, bf(*A), bf(*B), i32(OFF), with_weights=False)
    assert dx.shape == (10, 64) and da is None and db is None
    assert mgw.grouped_lora_backward(bf(10, 48), bf(*X), f32(10, 16), bf(*A), bf(*B), i32(OFF), with_dx=False)[0] is None


@pytest.mark.parametrize("bad", [
    dict(x=f32(*X)), dict(x=bf(10, 56)), dict(x=bf(64, 10).t()), dict(x=None), dict(a=bf(16, 64)), dict(a=f32(*A)),
    dict(b=bf(3, 48, 8)), dict(b=bf(2, 48, 16)), dict(b=f32(*B)), dict(adapter_off=i32(3)), dict(adapter_off=f32(OFF)),
    dict(scale=f32(2)), dict(scale=bf(3)), dict(row_index=f32(10)), dict(row_index=i32(5, 2)),
    dict(row_index=i32(10), out_index=i32(9)), dict(base=bf(10, 40)), dict(base=f32(10, 48)), dict(base=bf(9, 48)),
    dict(out_index=i32(11)), dict(row_index=i32(11), base=bf(10, 48)), dict(out=bf(10, 40)), dict(out=f32(10, 48)),
    dict(u=f32(10, 8)), dict(u=bf(10, 16)), dict(status=f32(1)),
], ids=str)
def test_lora_binding_refuses(fake, bad):
    args = dict(x=bf(*X), a=bf(*A), b=bf(*B), adapter_off=i32(OFF))
    with pytest.raises(mgw.MgwError):
        mgw.grouped_lora(**dict(args, **bad))
    assert fake.calls == []


@pytest.mark.parametrize("bad", [
    dict(dy=bf(10, 40)), dict(dy=f32(10, 48)), dict(x=None), dict(u=None), dict(x=bf(10, 56)), dict(x=bf(9, 64)),
    dict(u=f32(9, 16)), dict(u=bf(10, 16)), dict(dx_base=bf(10, 48)), dict(dx=bf(9, 64)), dict(da=f32(*A)),
    dict(db=bf(2, 48, 16)), dict(workspace=f32(64)), dict(workspace=torch.zeros(63, dtype=torch.uint8)),
    dict(with_dx=False, dx=bf(10, 64)), dict(with_weights=False, da=bf(*A)), dict(out_index=i32(10), row_index=i32(9)),
], ids=str)
def test_lora_backward_binding_refuses(fake, bad):
    args = dict(dy=bf(10, 48), x=bf(*X), u=f32(10, 16), a=bf(*A), b=bf(*B), adapter_off=i32(OFF))
    with pytest.raises(mgw.MgwError):
        mgw.grouped_lora_backward(**dict(args, **bad))
    assert fake.calls == []


def test_grad_shapes(fake):
    assert mgw.grad_norm([bf(3, 5), f32(7)]).shape == (1,)
    t = mgw.GradTable([bf(3, 5), f32(7), f32(0)], out=[bf(15), f32(7), f32(0)])
    assert mgw.clip_grads(t, 1.0).shape == (1,)
    known = f32(1)
    assert mgw.clip_grads([bf(4)], 1.0, known_norm=known) is known
    assert [c[0] for c in fake.calls] == ["mgw_grad_norm", "mgw_grad_clip", "mgw_grad_clip"]


def test_grad_binding_refuses(fake):
    a = bf(8)
    for grads, kw in (([torch.zeros(3, dtype=torch.float16)], {}), ([bf(4, 6).t()], {}), (["x"], {}), ([None], {}),
                      ([a], dict(norm=bf(1))), ([a], dict(norm=f32(0))), ([a], dict(workspace=f32(64))),
                      ([a], dict(workspace=torch.zeros(8, dtype=torch.uint8)))):
        for fn in (mgw.grad_norm, lambda g, **k: mgw.clip_grads(g, 1.0, **k)):
            with pytest.raises(mgw.MgwError):
                fn(grads, **kw)
    for bad in (lambda: mgw.clip_grads([a, a], 1.0), lambda: mgw.clip_grads([a], 1.0, known_norm=bf(1)),
                lambda: mgw.clip_grads([a], 1.0, known_norm=f32(1), norm=f32(1)), lambda: mgw.GradTable([a], out=[]),
                lambda: mgw.GradTable([a], out=[f32(8)]), lambda: mgw.GradTable([a], out=[bf(7)]),
                lambda: mgw.clip_grads(mgw.GradTable([bf(8), bf(8)], out=[a, a]), 1.0)):
        with pytest.raises(mgw.MgwError):
            bad()
    assert fake.calls == []
    mgw.grad_norm([a, a])   # a tensor may count twice


# (the call, tensors given, tensors it allocates)
CALLS = {
    "mgw_grouped_lora": (lambda **k: mgw.grouped_lora(bf(*X), bf(*A), bf(*B), i32(OFF), row_index=i32(10), out_index=i32(10),
                                                      scale=f32(3), base=bf(10, 48), save_u=True, **k), 8, 2),
    "mgw_grouped_lora_backward": (lambda **k: mgw.grouped_lora_backward(
        bf(10, 48), bf(*X), f32(10, 16), bf(*A), bf(*B), i32(OFF), scale=f32(3), dx_base=bf(10, 64), **k), 8, 4),
    "mgw_grad_norm": (lambda **k: mgw.grad_norm([bf(8), f32(3)], **k), 2, 2),
    "mgw_grad_clip": (lambda **k: mgw.clip_grads(mgw.GradTable([bf(8), f32(3)], out=[bf(8), f32(3)]), 1.0, **k), 4, 2),
}


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("which", ["side", "here", None])
def test_streams(fake, monkeypatch, name, which):
    """On another stream new memory comes from that stream's pool and every tensor is recorded on both;
    on the current one nothing is recorded."""
    here, side = FakeStream(0x10), FakeStream(0x20)
    now, allocated, recorded, keep = [here], [], [], []
    real_empty = torch.empty

    @contextlib.contextmanager
    def as_current(s):
        now.append(s)
        yield
        now.pop()

    def empty(*a, **k):
        keep.append(real_empty(*a, **k))
        allocated.append(now[-1])
        return keep[-1]

    call, given, made = CALLS[name]
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", as_current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *d: now[-1])
    monkeypatch.setattr(mgw, "_raw_stream", None)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: recorded.append((id(t), s)))
    call(stream={"side": side, "here": FakeStream(0x10), None: None}[which])
    assert [c[0] for c in fake.calls] == [name]
    if which == "side":
        assert allocated == [side] * made
        for s in (here, side):
            assert len({t for t, r in recorded if r is s}) == given + made
    else:
        assert allocated == [here] * made and recorded == []
