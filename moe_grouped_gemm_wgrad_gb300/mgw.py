"""Thin ctypes binding of libmgw.so (C ABI in include/mgw.h).

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  PyTorch provides device memory and the current stream.  If the
library is missing or fails to load, every call raises :class:`MgwError`;
there is no fallback implementation.

The C ABI sees only pointers, so the binding checks what the tensors know and the
library cannot: dtype, contiguity, one device for all operands, and that every
caller-supplied buffer holds at least the elements the call reads or writes.  A
failed check raises :class:`MgwError` before anything is launched.  Each call runs
with the operands' device current.

A call runs on the current stream, or on ``stream`` where that is given.  What it allocates
then belongs to ``stream``'s pool, and its tensors are recorded as in use on both streams,
so they may be dropped at any time.  Order between the streams is the caller's: ``stream``
has to wait for whoever writes the operands, and whoever reads the results for ``stream``.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmgw.so")
# The diagnostic build (include/mgw_diag.h): same results, plus a work-item timeline and
# device bounds checks.  Only diagnostic_library() switches the binding to it.
LIB_DIAG_PATH = os.path.join(HERE, "libmgw_diag.so")

MGW_OK = 0
MGW_DEV_BAD_OFFSETS = 1
MGW_DEV_TIMEOUT = 2
MGW_DEV_BAD_INDEX = 4
MGW_DEV_BOUNDS = 8   # diagnostic library only
MGW_DEV_BAD_LOGIT = 16
DIAG_KERNELS = {1: "grouped_wgrad_pair_kernel", 2: "grouped_dgrad_kernel", 3: "grouped_dgrad_pair_kernel"}
MAX_EXPERTS = 1024
SCALE_FLOOR = 0      # OCP MX rule 2^(floor(log2 amax) - 8)
SCALE_CEIL_448 = 1   # the post-attn page's RoundUp rule ceil_pow2(amax / 448)
TYPE_BF16 = 0
TYPE_F32 = 1
SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
ACT_NONE = 0
ACT_RELU = 1
ACT_GELU = 2         # x * Phi(x)
ACT_SILU = 3
ACT_SWIGLU = 4       # silu(gate) * up, the product's columns being gate then up
ACT_GEGLU = 5        # gelu(gate) * up
GATED_ACTS = (ACT_SWIGLU, ACT_GEGLU)
MAX_TOP_K = 32
MAX_RANK = 128       # of a low-rank adapter
MAX_SIZE = 2 ** 31 - 1   # of every size and count in the C ABI

EXPORTS = (
    "mgw_status_string", "mgw_version", "mgw_mxfp8_token_capacity", "mgw_mxfp8_scale_bytes",
    "mgw_mxfp8_quantize", "mgw_mxfp8_quantize_gather", "mgw_grouped_wgrad_mxfp8",
    "mgw_grouped_dgrad_f32", "mgw_mxfp8_quantize_rows", "mgw_grouped_fprop_mxfp8",
    "mgw_grouped_dgrad_mxfp8", "mgw_grouped_wgrad_mxfp8_balanced",
    "mgw_grouped_wgrad_workspace_bytes", "mgw_grouped_wgrad_mxfp8_balanced_noalloc",
    "mgw_moe_route", "mgw_moe_route_backward", "mgw_moe_dispatch",
    "mgw_moe_dispatch_workspace_bytes", "mgw_grouped_fprop_mxfp8_act", "mgw_grouped_act_backward",
    "mgw_grouped_act_backward_workspace_bytes", "mgw_moe_combine", "mgw_moe_combine_backward",
    "mgw_grouped_lora", "mgw_grouped_lora_backward", "mgw_grouped_lora_backward_workspace_bytes",
    "mgw_grad_norm", "mgw_grad_clip", "mgw_grad_workspace_bytes",
)


DIAG_EXPORTS = ("mgw_diag_timeline", "mgw_diag_timeline_reset")


class MgwError(RuntimeError):
    pass


class DiagRecord(ctypes.Structure):
    """mgw_diag_record of include/mgw_diag.h."""
    _fields_ = [("kernel", ctypes.c_uint32), ("sm", ctypes.c_uint32), ("cta", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("item", ctypes.c_int64),
                ("t_wait_ns", ctypes.c_uint64), ("t_done_ns", ctypes.c_uint64)]


_lock = threading.Lock()
_lib = None


def bind(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Declares the C ABI's argument and return types on a loaded build of the library."""
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.mgw_status_string.argtypes = [I]
    lib.mgw_status_string.restype = ctypes.c_char_p
    lib.mgw_version.argtypes = []
    lib.mgw_version.restype = I
    lib.mgw_mxfp8_token_capacity.argtypes = [I, I]
    lib.mgw_mxfp8_token_capacity.restype = SZ
    lib.mgw_mxfp8_scale_bytes.argtypes = [I, SZ]
    lib.mgw_mxfp8_scale_bytes.restype = SZ
    lib.mgw_mxfp8_quantize.argtypes = [P, I, I, P, I, P, P, SZ, I, P, P]
    lib.mgw_mxfp8_quantize.restype = I
    lib.mgw_mxfp8_quantize_gather.argtypes = [P, I, P, I, I, P, I, P, P, SZ, I, P, P]
    lib.mgw_mxfp8_quantize_gather.restype = I
    lib.mgw_grouped_wgrad_mxfp8.argtypes = [P, P, P, P, P, I, I, I, I, SZ, P, P, P]
    lib.mgw_grouped_wgrad_mxfp8.restype = I
    lib.mgw_grouped_dgrad_f32.argtypes = [P, P, P, I, I, I, I, P, P, P]
    lib.mgw_grouped_dgrad_f32.restype = I
    lib.mgw_mxfp8_quantize_rows.argtypes = [P, I, P, I, I, P, I, P, P, SZ, I, P, P]
    lib.mgw_mxfp8_quantize_rows.restype = I
    lib.mgw_grouped_fprop_mxfp8.argtypes = [P, P, P, P, P, I, I, I, I, SZ, SZ, P, P, P]
    lib.mgw_grouped_fprop_mxfp8.restype = I
    lib.mgw_grouped_dgrad_mxfp8.argtypes = [P, P, P, P, P, I, I, I, I, SZ, SZ, P, P, P]
    lib.mgw_grouped_dgrad_mxfp8.restype = I
    lib.mgw_grouped_wgrad_mxfp8_balanced.argtypes = [P, P, P, P, P, I, I, I, I, SZ, P, P, SZ, P, P]
    lib.mgw_grouped_wgrad_mxfp8_balanced.restype = I
    lib.mgw_grouped_wgrad_workspace_bytes.argtypes = [I, I, I]
    lib.mgw_grouped_wgrad_workspace_bytes.restype = SZ
    lib.mgw_grouped_wgrad_mxfp8_balanced_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, SZ, P, P, P]
    lib.mgw_grouped_wgrad_mxfp8_balanced_noalloc.restype = I
    FL = ctypes.c_float
    lib.mgw_moe_route.argtypes = [P, I, I, I, P, I, I, I, I, I, I, FL, P, P, P, P, P]
    lib.mgw_moe_route.restype = I
    lib.mgw_moe_route_backward.argtypes = [P, I, I, I, I, I, I, FL, P, P, P, P, P, P]
    lib.mgw_moe_route_backward.restype = I
    lib.mgw_moe_dispatch.argtypes = [P, I, I, I, P, P, P, P, SZ, P, P]
    lib.mgw_moe_dispatch.restype = I
    lib.mgw_moe_dispatch_workspace_bytes.argtypes = [I, I, I]
    lib.mgw_moe_dispatch_workspace_bytes.restype = SZ
    lib.mgw_grouped_fprop_mxfp8_act.argtypes = [P, P, P, P, P, I, I, I, I, SZ, SZ, I, P, P, P, P, P, P]
    lib.mgw_grouped_fprop_mxfp8_act.restype = I
    lib.mgw_grouped_act_backward.argtypes = [P, P, P, I, I, I, I, P, P, P, SZ, P, P]
    lib.mgw_grouped_act_backward.restype = I
    lib.mgw_grouped_act_backward_workspace_bytes.argtypes = [I, I, I]
    lib.mgw_grouped_act_backward_workspace_bytes.restype = SZ
    lib.mgw_moe_combine.argtypes = [P, I, I, P, P, P, I, I, I, P, P, P]
    lib.mgw_moe_combine.restype = I
    lib.mgw_moe_combine_backward.argtypes = [P, P, I, I, P, P, I, I, I, P, P, P, P]
    lib.mgw_moe_combine_backward.restype = I
    lib.mgw_grouped_lora.argtypes = [P, I, P, I, I, P, P, P, P, I, I, I, P, P, I, P, P, P, P]
    lib.mgw_grouped_lora.restype = I
    lib.mgw_grouped_lora_backward.argtypes = [P, I, P, P, I, P, I, I, P, P, P, P, I, I, I, P, P, P, P, P, P, SZ,
                                              P, P]
    lib.mgw_grouped_lora_backward.restype = I
    lib.mgw_grouped_lora_backward_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.mgw_grouped_lora_backward_workspace_bytes.restype = SZ
    lib.mgw_grad_norm.argtypes = [P, P, P, I, P, P, SZ, P]
    lib.mgw_grad_norm.restype = I
    lib.mgw_grad_clip.argtypes = [P, P, P, P, I, FL, FL, P, P, P, SZ, P]
    lib.mgw_grad_clip.restype = I
    lib.mgw_grad_workspace_bytes.argtypes = [I]
    lib.mgw_grad_workspace_bytes.restype = SZ
    return lib


def bind_diag(lib: ctypes.CDLL) -> ctypes.CDLL:
    """bind() plus the two entry points only the diagnostic library exports."""
    bind(lib)
    lib.mgw_diag_timeline.argtypes = [ctypes.POINTER(DiagRecord), ctypes.c_int,
                                      ctypes.POINTER(ctypes.c_int)]
    lib.mgw_diag_timeline.restype = ctypes.c_int
    lib.mgw_diag_timeline_reset.argtypes = []
    lib.mgw_diag_timeline_reset.restype = ctypes.c_int
    return lib


_diag_lib = None


@contextlib.contextmanager
def diagnostic_library():
    """Runs the calls made inside the block through libmgw_diag.so (built beside libmgw.so):
    the same results, a work-item timeline (diag_timeline) and device bounds checks that set
    MGW_DEV_BOUNDS in a call's status word.  Not thread-safe against concurrent calls made
    outside the block."""
    global _lib, _diag_lib
    with _lock:
        if _diag_lib is None:
            if not os.path.exists(LIB_DIAG_PATH):
                raise MgwError(f"{LIB_DIAG_PATH} is not built; run `python -m moe_grouped_gemm_wgrad_gb300.build`")
            _diag_lib = bind_diag(ctypes.CDLL(LIB_DIAG_PATH))
        prev, _lib = _lib, _diag_lib
    try:
        yield _diag_lib
    finally:
        with _lock:
            _lib = prev


def diag_timeline(cap: int = 3 * 65536) -> list[dict]:
    """The work-item timeline recorded by the diagnostic library since the last
    diag_timeline_reset(), one dict per (CTA, item); synchronises with the device."""
    if _diag_lib is None:
        raise MgwError("diag_timeline needs diagnostic_library() to have been entered")
    buf = (DiagRecord * cap)()
    total = ctypes.c_int(0)
    _check(_diag_lib.mgw_diag_timeline(buf, cap, ctypes.byref(total)), "mgw_diag_timeline")
    out = []
    for r in buf[:min(cap, total.value)]:
        out.append({"kernel": DIAG_KERNELS.get(r.kernel, str(r.kernel)), "sm": r.sm, "cta": r.cta,
                    "item": r.item, "t_wait_ns": r.t_wait_ns, "t_done_ns": r.t_done_ns})
    return out


def diag_timeline_reset() -> None:
    if _diag_lib is None:
        raise MgwError("diag_timeline_reset needs diagnostic_library() to have been entered")
    _check(_diag_lib.mgw_diag_timeline_reset(), "mgw_diag_timeline_reset")


def load() -> ctypes.CDLL:
    """Load libmgw.so (built in-tree by ``moe_grouped_gemm_wgrad_gb300.build``)."""
    global _lib
    lib = _lib
    if lib is not None:
        return lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise MgwError(f"{LIB_PATH} is not built; run `python -m moe_grouped_gemm_wgrad_gb300.build`")
        _lib = bind(ctypes.CDLL(LIB_PATH))
        return _lib


def _check(st: int, what: str) -> None:
    if st != MGW_OK:
        msg = load().mgw_status_string(st).decode()
        raise MgwError(f"{what}: {msg} (status {st})")


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


# torch's raw handle of a device's current stream: 0.2 us, where the public Stream object takes 2.9.
# A torch without it goes through that object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    """The raw handle of ``stream``, or of the current device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(torch.cuda.current_device())


def _on_cuda(t: torch.Tensor) -> bool:
    return t.is_cuda


def _dev_tensor(t: torch.Tensor, dtype, name: str, ndim: int | None = None) -> None:
    if not isinstance(t, torch.Tensor) or not _on_cuda(t):
        raise MgwError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise MgwError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise MgwError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise MgwError(f"{name} must be {ndim}-D, got shape {tuple(t.shape)}")
    if t.numel() > MAX_SIZE and max(t.shape) > MAX_SIZE:
        raise MgwError(f"a dimension of {name} {tuple(t.shape)} exceeds the C ABI's 32-bit sizes")


def _size(n, name: str) -> int:
    """``n`` as a size that the C ABI's 32-bit arguments hold (ctypes would cut it down silently)."""
    n = int(n)
    if n > MAX_SIZE or n < -MAX_SIZE:
        raise MgwError(f"{name} = {n} exceeds the C ABI's 32-bit sizes")
    return n


def _need(t: torch.Tensor, n: int, name: str) -> None:
    """``t`` holds at least the ``n`` elements the call touches."""
    if t.numel() < n:
        raise MgwError(f"{name} holds {t.numel()} elements; the call needs {n}")


def _offsets(expert_off: torch.Tensor, E: int | None = None) -> int:
    """Checks expert_off (int32, E+1 >= 2 entries) and returns E."""
    _dev_tensor(expert_off, torch.int32, "expert_off", 1)
    n = expert_off.numel()
    if n < 2:
        raise MgwError("expert_off needs E+1 >= 2 entries")
    if E is not None and n != E + 1:
        raise MgwError(f"expert_off has {n} entries; {E} experts need {E + 1}")
    return n - 1


def _status(status: torch.Tensor | None) -> None:
    if status is not None:
        _dev_tensor(status, torch.int32, "status")
        _need(status, 1, "status")


def _one_device(*ts) -> torch.device:
    first = None
    for t in ts:
        if t is None:
            continue
        if first is None:
            first, dev = t, t.device
        elif t.device != dev:
            devs = {str(u.device) for u in ts if u is not None}
            raise MgwError(f"all tensors must be on one CUDA device, got {sorted(devs)}")
    return dev


def _out(t: torch.Tensor | None, shape, dtype, dev, name: str, side=None) -> torch.Tensor:
    """The caller's output or workspace buffer after checks, or a new one of ``shape``: from the pool
    of the stream ``side`` that the call runs on, if that is not the current one.  Memory of the
    current stream's pool may still be in use by work queued there, for which ``side`` does not wait."""
    if t is None:
        if side is None:
            return torch.empty(shape, dtype=dtype, device=dev)
        with torch.cuda.stream(side):
            return torch.empty(shape, dtype=dtype, device=dev)
    n = 1
    for d in shape:
        n *= int(d)
    _dev_tensor(t, dtype, name)
    _need(t, n, name)
    return t


_AS_IT_IS = contextlib.nullcontext()


def _device(dev: torch.device):
    """Makes ``dev`` the current CUDA device for the call (the library launches on, and
    sizes its grids for, the current device)."""
    if torch.cuda.current_device() == dev.index:
        return _AS_IT_IS
    return torch.cuda.device(dev)


def _side(stream, dev: torch.device):
    """``stream`` as a torch stream where it is not ``dev``'s current one, else None."""
    handle = stream.cuda_stream
    here = torch.cuda.current_stream(dev).cuda_stream if _raw_stream is None else _raw_stream(dev.index)
    if handle == here:
        return None
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(handle, device=dev)


def _used_on(side, *ts) -> None:
    """Tells the allocator that the tensors of a call on ``side`` are in use there and on the current
    stream, so that memory that the host frees meanwhile is handed out again only when both streams
    are past this point."""
    for t in ts:
        if t is not None:
            t.record_stream(side)
            t.record_stream(torch.cuda.current_stream(t.device))


def token_capacity(M: int, E: int) -> int:
    """Padded token axis length that fits any split of M tokens over E experts."""
    return int(load().mgw_mxfp8_token_capacity(_size(M, "M"), _size(E, "E")))


def scale_bytes(C: int, Mcap: int) -> int:
    return int(load().mgw_mxfp8_scale_bytes(int(C), int(Mcap)))


def mxfp8_quantize(src: torch.Tensor, expert_off: torch.Tensor, Mcap: int | None = None,
                   q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                   status: torch.Tensor | None = None, stream=None, scale_rule: int = SCALE_FLOOR):
    """MXFP8-quantize bf16 ``src`` [M, C] along tokens -> (q uint8 [C, Mcap], scales uint8)."""
    _dev_tensor(src, torch.bfloat16, "src", 2)
    E = _offsets(expert_off)
    _status(status)
    M, C = src.shape
    Mcap = token_capacity(M, E) if Mcap is None else int(Mcap)
    dev = _one_device(src, expert_off, q, scales, status)
    side = None if stream is None else _side(stream, dev)
    q = _out(q, (C, Mcap), torch.uint8, dev, "q", side)
    scales = _out(scales, (scale_bytes(C, Mcap),), torch.uint8, dev, "scales", side)
    with _device(dev):
        st = load().mgw_mxfp8_quantize(_ptr(src), M, C, _ptr(expert_off), E, _ptr(q), _ptr(scales),
                                       Mcap, int(scale_rule), _ptr(status), _stream(stream))
    _check(st, "mgw_mxfp8_quantize")
    if side is not None:
        _used_on(side, src, expert_off, q, scales, status)
    return q, scales


def mxfp8_quantize_gather(src: torch.Tensor, row_index: torch.Tensor, expert_off: torch.Tensor,
                          Mcap: int | None = None, q: torch.Tensor | None = None,
                          scales: torch.Tensor | None = None, status: torch.Tensor | None = None,
                          stream=None, scale_rule: int = SCALE_FLOOR):
    """MXFP8-quantize the routed rows src[row_index] (src bf16 [rows, C], row_index int32 [M])
    without materialising them -> (q uint8 [C, Mcap], scales uint8)."""
    _dev_tensor(src, torch.bfloat16, "src", 2)
    _dev_tensor(row_index, torch.int32, "row_index", 1)
    E = _offsets(expert_off)
    _status(status)
    src_rows, C = src.shape
    M = row_index.numel()
    Mcap = token_capacity(M, E) if Mcap is None else int(Mcap)
    dev = _one_device(src, row_index, expert_off, q, scales, status)
    side = None if stream is None else _side(stream, dev)
    q = _out(q, (C, Mcap), torch.uint8, dev, "q", side)
    scales = _out(scales, (scale_bytes(C, Mcap),), torch.uint8, dev, "scales", side)
    with _device(dev):
        st = load().mgw_mxfp8_quantize_gather(_ptr(src), src_rows, _ptr(row_index), M, C,
                                              _ptr(expert_off), E, _ptr(q), _ptr(scales), Mcap,
                                              int(scale_rule), _ptr(status), _stream(stream))
    _check(st, "mgw_mxfp8_quantize_gather")
    if side is not None:
        _used_on(side, src, row_index, expert_off, q, scales, status)
    return q, scales


def _wgrad_operands(gq, gs, xq, xs, expert_off, status, *others):
    """Checks the quantized wgrad operands; returns (E, N, K, Mcap, device)."""
    for t, n in ((gq, "gq"), (xq, "xq")):
        _dev_tensor(t, torch.uint8, n, 2)
    for t, n in ((gs, "gs"), (xs, "xs")):
        _dev_tensor(t, torch.uint8, n)
    E = _offsets(expert_off)
    _status(status)
    N, Mcap = gq.shape
    K, Mcap_x = xq.shape
    if Mcap_x != Mcap:
        raise MgwError(f"gq [N, {Mcap}] and xq [K, {Mcap_x}] must share one padded token axis")
    _need(gs, scale_bytes(N, Mcap), "gs")
    _need(xs, scale_bytes(K, Mcap), "xs")
    dev = _one_device(gq, gs, xq, xs, expert_off, status, *others)
    return E, N, K, Mcap, dev


def grouped_wgrad_mxfp8(gq: torch.Tensor, gs: torch.Tensor, xq: torch.Tensor, xs: torch.Tensor,
                        expert_off: torch.Tensor, M: int, out: torch.Tensor | None = None,
                        status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """grad_w [E*N, K] bf16 from quantized g^T (N rows) and x^T (K rows)."""
    E, N, K, Mcap, dev = _wgrad_operands(gq, gs, xq, xs, expert_off, status, out)
    side = None if stream is None else _side(stream, dev)
    M = _size(M, "M")
    out = _out(out, (E * N, K), torch.bfloat16, dev, "out", side)
    with _device(dev):
        st = load().mgw_grouped_wgrad_mxfp8(_ptr(gq), _ptr(gs), _ptr(xq), _ptr(xs),
                                            _ptr(expert_off), E, M, N, K, Mcap, _ptr(out),
                                            _ptr(status), _stream(stream))
    _check(st, "mgw_grouped_wgrad_mxfp8")
    if side is not None:
        _used_on(side, gq, gs, xq, xs, expert_off, out, status)
    return out


def wgrad_workspace(E: int, N: int, K: int, device=None) -> torch.Tensor:
    """A zero-filled workspace for :func:`grouped_wgrad_mxfp8_balanced` on ``device``."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(dev):
        nbytes = int(load().mgw_grouped_wgrad_workspace_bytes(_size(E, "E"), _size(N, "N"), _size(K, "K")))
    if nbytes == 0:
        raise MgwError("mgw_grouped_wgrad_workspace_bytes: no usable device")
    return torch.zeros(nbytes, dtype=torch.uint8, device=dev)


def grouped_wgrad_mxfp8_balanced(gq: torch.Tensor, gs: torch.Tensor, xq: torch.Tensor,
                                 xs: torch.Tensor, expert_off: torch.Tensor, M: int,
                                 workspace: torch.Tensor, out: torch.Tensor | None = None,
                                 status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """grad_w [E*N, K] bf16, as :func:`grouped_wgrad_mxfp8`, with split-K and dynamic
    scheduling for skewed routings.  ``workspace``: uint8, zero-filled before first use
    (see :func:`wgrad_workspace`); calls sharing it must not overlap."""
    _dev_tensor(workspace, torch.uint8, "workspace")
    E, N, K, Mcap, dev = _wgrad_operands(gq, gs, xq, xs, expert_off, status, out, workspace)
    side = None if stream is None else _side(stream, dev)
    M = _size(M, "M")
    out = _out(out, (E * N, K), torch.bfloat16, dev, "out", side)
    with _device(dev):
        st = load().mgw_grouped_wgrad_mxfp8_balanced(
            _ptr(gq), _ptr(gs), _ptr(xq), _ptr(xs), _ptr(expert_off), E, M, N, K, Mcap,
            _ptr(out), _ptr(workspace), workspace.numel(), _ptr(status), _stream(stream))
    _check(st, "mgw_grouped_wgrad_mxfp8_balanced")
    if side is not None:
        _used_on(side, gq, gs, xq, xs, expert_off, workspace, out, status)
    return out


def grouped_wgrad_mxfp8_balanced_noalloc(gq: torch.Tensor, gs: torch.Tensor, xq: torch.Tensor,
                                         xs: torch.Tensor, expert_off: torch.Tensor, M: int,
                                         out: torch.Tensor | None = None,
                                         status: torch.Tensor | None = None,
                                         stream=None) -> torch.Tensor:
    """As :func:`grouped_wgrad_mxfp8_balanced` on the library's own workspace (a device array
    in the library; nothing is allocated, calls must not overlap)."""
    E, N, K, Mcap, dev = _wgrad_operands(gq, gs, xq, xs, expert_off, status, out)
    side = None if stream is None else _side(stream, dev)
    M = _size(M, "M")
    out = _out(out, (E * N, K), torch.bfloat16, dev, "out", side)
    with _device(dev):
        st = load().mgw_grouped_wgrad_mxfp8_balanced_noalloc(
            _ptr(gq), _ptr(gs), _ptr(xq), _ptr(xs), _ptr(expert_off), E, M, N, K, Mcap,
            _ptr(out), _ptr(status), _stream(stream))
    _check(st, "mgw_grouped_wgrad_mxfp8_balanced_noalloc")
    if side is not None:
        _used_on(side, gq, gs, xq, xs, expert_off, out, status)
    return out


def grouped_dgrad_f32(dy: torch.Tensor, W: torch.Tensor, expert_off: torch.Tensor,
                      out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """dx [rows, in_f] fp32 = dy[r] . W[e(r)] per row's expert."""
    _dev_tensor(dy, torch.float32, "dy", 2)
    _dev_tensor(W, torch.float32, "W", 3)
    rows, out_f = dy.shape
    E, out_w, in_f = W.shape
    if out_w != out_f:
        raise MgwError(f"W [E, {out_w}, in_f] does not match dy [rows, {out_f}]")
    _offsets(expert_off, E)
    _status(status)
    dev = _one_device(dy, W, expert_off, out, status)
    side = None if stream is None else _side(stream, dev)
    out = _out(out, (rows, in_f), torch.float32, dev, "out", side)
    with _device(dev):
        st = load().mgw_grouped_dgrad_f32(_ptr(dy), _ptr(W), _ptr(expert_off), E, rows, out_f,
                                          in_f, _ptr(out), _ptr(status), _stream(stream))
    _check(st, "mgw_grouped_dgrad_f32")
    if side is not None:
        _used_on(side, dy, W, expert_off, out, status)
    return out


def mxfp8_quantize_rows(src: torch.Tensor, expert_off: torch.Tensor, Mcap: int | None = None,
                        q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                        status: torch.Tensor | None = None, stream=None,
                        scale_rule: int = SCALE_FLOOR, row_index: torch.Tensor | None = None):
    """Row-wise MXFP8 quantization (one scale per 32 columns of a row) of the routed rows:
    ``src[row_index]`` when ``row_index`` (int32 [M]) is given, else ``src`` [M, C].
    -> (q uint8 [Mcap, C] on the padded row axis, scale atoms uint8)."""
    _dev_tensor(src, torch.bfloat16, "src", 2)
    E = _offsets(expert_off)
    _status(status)
    src_rows, C = src.shape
    if row_index is not None:
        _dev_tensor(row_index, torch.int32, "row_index", 1)
        M = row_index.numel()
    else:
        M = src_rows
    Mcap = token_capacity(M, E) if Mcap is None else int(Mcap)
    dev = _one_device(src, expert_off, row_index, q, scales, status)
    side = None if stream is None else _side(stream, dev)
    q = _out(q, (Mcap, C), torch.uint8, dev, "q", side)
    scales = _out(scales, (scale_bytes(C, Mcap),), torch.uint8, dev, "scales", side)
    with _device(dev):
        st = load().mgw_mxfp8_quantize_rows(_ptr(src), src_rows, _ptr(row_index), M, C,
                                            _ptr(expert_off), E, _ptr(q), _ptr(scales), Mcap,
                                            int(scale_rule), _ptr(status), _stream(stream))
    _check(st, "mgw_mxfp8_quantize_rows")
    if side is not None:
        _used_on(side, src, expert_off, row_index, q, scales, status)
    return q, scales


def grouped_fprop_mxfp8(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor, ws: torch.Tensor,
                        expert_off: torch.Tensor, M: int, N: int, out: torch.Tensor | None = None,
                        status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [M, N] bf16 = x[r] . W[e(r)]^T from row-wise quantized x [Mcap, K] and W [Mw, K]
    (W [E, N, K] quantized with offsets {0, N, ..., E*N})."""
    for t, n in ((xq, "xq"), (wq, "wq")):
        _dev_tensor(t, torch.uint8, n, 2)
    for t, n in ((xs, "xs"), (ws, "ws")):
        _dev_tensor(t, torch.uint8, n)
    E = _offsets(expert_off)
    _status(status)
    Mcap, K = xq.shape
    Mw, K_w = wq.shape
    if K_w != K:
        raise MgwError(f"wq [Mw, {K_w}] and xq [Mcap, {K}] must share the contraction width")
    _need(xs, scale_bytes(K, Mcap), "xs")
    _need(ws, scale_bytes(K, Mw), "ws")
    dev = _one_device(xq, xs, wq, ws, expert_off, out, status)
    side = None if stream is None else _side(stream, dev)
    M, N = _size(M, "M"), _size(N, "N")
    out = _out(out, (M, N), torch.bfloat16, dev, "out", side)
    with _device(dev):
        st = load().mgw_grouped_fprop_mxfp8(_ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws),
                                            _ptr(expert_off), E, M, N, K, Mcap, Mw,
                                            _ptr(out), _ptr(status), _stream(stream))
    _check(st, "mgw_grouped_fprop_mxfp8")
    if side is not None:
        _used_on(side, xq, xs, wq, ws, expert_off, out, status)
    return out


def grouped_dgrad_mxfp8(dyq: torch.Tensor, dys: torch.Tensor, wtq: torch.Tensor,
                        wts: torch.Tensor, expert_off: torch.Tensor, M: int,
                        out: torch.Tensor | None = None, status: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """dx [M, K] bf16 = dy[r] . W[e(r)] from row-wise quantized dy [Mcap, N] and W quantized
    along n per expert by :func:`mxfp8_quantize` (wtq [K, Mw])."""
    for t, n in ((dyq, "dyq"), (wtq, "wtq")):
        _dev_tensor(t, torch.uint8, n, 2)
    for t, n in ((dys, "dys"), (wts, "wts")):
        _dev_tensor(t, torch.uint8, n)
    E = _offsets(expert_off)
    _status(status)
    Mcap, N = dyq.shape
    K, Mw = wtq.shape
    _need(dys, scale_bytes(N, Mcap), "dys")
    _need(wts, scale_bytes(K, Mw), "wts")
    dev = _one_device(dyq, dys, wtq, wts, expert_off, out, status)
    side = None if stream is None else _side(stream, dev)
    M = _size(M, "M")
    out = _out(out, (M, K), torch.bfloat16, dev, "out", side)
    with _device(dev):
        st = load().mgw_grouped_dgrad_mxfp8(_ptr(dyq), _ptr(dys), _ptr(wtq), _ptr(wts),
                                            _ptr(expert_off), E, M, N, K, Mcap, Mw,
                                            _ptr(out), _ptr(status), _stream(stream))
    _check(st, "mgw_grouped_dgrad_mxfp8")
    if side is not None:
        _used_on(side, dyq, dys, wtq, wts, expert_off, out, status)
    return out


# ------------------------------------------------------------------- the routed layer
def _element_type(t: torch.Tensor, name: str) -> int:
    """The C ABI's code of a bf16 or fp32 tensor's type."""
    if not isinstance(t, torch.Tensor):
        raise MgwError(f"{name} must be a CUDA tensor")
    if t.dtype == torch.bfloat16:
        return TYPE_BF16
    if t.dtype == torch.float32:
        return TYPE_F32
    raise MgwError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")


def _shaped(t: torch.Tensor, shape, dtype, name: str) -> None:
    """``t`` is a contiguous device tensor of exactly ``shape``."""
    _dev_tensor(t, dtype, name, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise MgwError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")


def moe_route(logits: torch.Tensor, top_k: int, bias: torch.Tensor | None = None,
              score: int = SCORE_SOFTMAX, groups: int = 1, top_groups: int = 1,
              group_best: int = 1, renorm: bool = True, scale: float = 1.0,
              with_scores: bool = False, expert_idx: torch.Tensor | None = None,
              weights: torch.Tensor | None = None, scores: torch.Tensor | None = None,
              status: torch.Tensor | None = None, stream=None):
    """The top_k experts of every token of ``logits`` [T, E] (bf16 or fp32) and their weights
    -> (expert_idx int32 [T, top_k], weights fp32 [T, top_k]), and the scores fp32 [T, E] as a
    third value when ``with_scores`` (or ``scores``) is given.

    ``bias`` (fp32 [E]) moves the choice but not the weights.  With ``groups`` > 1 only experts
    of the ``top_groups`` best of ``groups`` equal runs can be chosen, a run's value being its
    best expert's or (``group_best`` 2) the sum of its two best.  Logits of -inf are masked;
    slots that no expert is left for hold -1 with weight 0."""
    dt = _element_type(logits, "logits")
    _dev_tensor(logits, logits.dtype, "logits", 2)
    T, E = logits.shape
    top_k = _size(top_k, "top_k")
    if top_k < 1 or top_k > min(MAX_TOP_K, E):
        raise MgwError(f"top_k must be 1 .. {min(MAX_TOP_K, E)}, got {top_k}")
    if bias is not None:
        _shaped(bias, (E,), torch.float32, "bias")
    _status(status)
    dev = _one_device(logits, bias, expert_idx, weights, scores, status)
    side = None if stream is None else _side(stream, dev)
    expert_idx = _out(expert_idx, (T, top_k), torch.int32, dev, "expert_idx", side)
    weights = _out(weights, (T, top_k), torch.float32, dev, "weights", side)
    if with_scores or scores is not None:
        scores = _out(scores, (T, E), torch.float32, dev, "scores", side)
    with _device(dev):
        st = load().mgw_moe_route(_ptr(logits), dt, T, E, _ptr(bias), top_k, int(score),
                                  int(groups), int(top_groups), int(group_best), int(bool(renorm)),
                                  float(scale), _ptr(expert_idx), _ptr(weights), _ptr(scores),
                                  _ptr(status), _stream(stream))
    _check(st, "mgw_moe_route")
    if side is not None:
        _used_on(side, logits, bias, expert_idx, weights, scores, status)
    return (expert_idx, weights) if scores is None else (expert_idx, weights, scores)


def moe_route_backward(logits: torch.Tensor, expert_idx: torch.Tensor,
                       dweights: torch.Tensor | None, dscores: torch.Tensor | None = None,
                       score: int = SCORE_SOFTMAX, renorm: bool = True, scale: float = 1.0,
                       dlogits: torch.Tensor | None = None, status: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """dlogits [T, E] (the logits' type) from the gradients of :func:`moe_route`'s weights and,
    when the scores are used too, of its scores.  ``logits``, ``expert_idx``, ``score``,
    ``renorm`` and ``scale`` as in the forward call."""
    dt = _element_type(logits, "logits")
    _dev_tensor(logits, logits.dtype, "logits", 2)
    T, E = logits.shape
    _dev_tensor(expert_idx, torch.int32, "expert_idx", 2)
    top_k = expert_idx.shape[1]
    _shaped(expert_idx, (T, top_k), torch.int32, "expert_idx")
    if dweights is not None:
        _shaped(dweights, (T, top_k), torch.float32, "dweights")
    if dscores is not None:
        _shaped(dscores, (T, E), torch.float32, "dscores")
    _status(status)
    dev = _one_device(logits, expert_idx, dweights, dscores, dlogits, status)
    side = None if stream is None else _side(stream, dev)
    dlogits = _out(dlogits, (T, E), logits.dtype, dev, "dlogits", side)
    with _device(dev):
        st = load().mgw_moe_route_backward(_ptr(logits), dt, T, E, top_k, int(score),
                                           int(bool(renorm)), float(scale), _ptr(expert_idx),
                                           _ptr(dweights), _ptr(dscores), _ptr(dlogits),
                                           _ptr(status), _stream(stream))
    _check(st, "mgw_moe_route_backward")
    if side is not None:
        _used_on(side, logits, expert_idx, dweights, dscores, dlogits, status)
    return dlogits


def moe_dispatch(expert_idx: torch.Tensor, E: int, expert_off: torch.Tensor | None = None,
                 row_index: torch.Tensor | None = None, row_of: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                 stream=None):
    """The row tables of a routing ``expert_idx`` int32 [T, top_k] (-1: dropped) over E experts
    -> (expert_off int32 [E+1], row_index int32 [T*top_k], row_of int32 [T, top_k]).

    ``expert_off`` and ``row_index`` are what the quantizers and grouped products take, with
    M = expert_off[E] rows: T * top_k when nothing is dropped.  Where pairs may be dropped, read
    ``M = int(expert_off[-1])`` back (these calls take M from the host) and pass
    ``row_index[:M]``.  ``row_of`` is what :func:`moe_combine` takes.  ``workspace`` (uint8) is allocated when a large call needs one
    and none is given."""
    _dev_tensor(expert_idx, torch.int32, "expert_idx", 2)
    T, top_k = expert_idx.shape
    E = _size(E, "E")
    if E < 1:
        raise MgwError(f"E must be at least 1, got {E}")
    _status(status)
    dev = _one_device(expert_idx, expert_off, row_index, row_of, workspace, status)
    lib = load()
    need = int(lib.mgw_moe_dispatch_workspace_bytes(T, top_k, E))
    side = None if stream is None else _side(stream, dev)
    workspace = _out(workspace, (need,), torch.uint8, dev, "workspace", side) \
        if need or workspace is not None else None
    expert_off = _out(expert_off, (E + 1,), torch.int32, dev, "expert_off", side)
    row_index = _out(row_index, (T * top_k,), torch.int32, dev, "row_index", side)
    row_of = _out(row_of, (T, top_k), torch.int32, dev, "row_of", side)
    with _device(dev):
        st = lib.mgw_moe_dispatch(_ptr(expert_idx), T, top_k, E, _ptr(expert_off), _ptr(row_index),
                                  _ptr(row_of), _ptr(workspace),
                                  0 if workspace is None else workspace.numel(), _ptr(status),
                                  _stream(stream))
    _check(st, "mgw_moe_dispatch")
    if side is not None:
        _used_on(side, expert_idx, expert_off, row_index, row_of, workspace, status)
    return expert_off, row_index, row_of


def grouped_fprop_mxfp8_act(xq: torch.Tensor, xs: torch.Tensor, wq: torch.Tensor,
                            ws: torch.Tensor, expert_off: torch.Tensor, M: int, N: int,
                            act: int = ACT_NONE, bias: torch.Tensor | None = None,
                            residual: torch.Tensor | None = None, save_preact: bool = False,
                            out: torch.Tensor | None = None, preact: torch.Tensor | None = None,
                            status: torch.Tensor | None = None, stream=None):
    """y [M, F] bf16 = act(x[r] . W[e(r)]^T + bias[e(r)]) + residual, F = N (N / 2 for the gated
    activations, whose gate columns come first), from the operands of
    :func:`grouped_fprop_mxfp8`.  With ``save_preact`` (or ``preact``) returns (y, z), z [M, N]
    bf16 being the pre-activation that :func:`grouped_act_backward` takes."""
    for t, n in ((xq, "xq"), (wq, "wq")):
        _dev_tensor(t, torch.uint8, n, 2)
    for t, n in ((xs, "xs"), (ws, "ws")):
        _dev_tensor(t, torch.uint8, n)
    E = _offsets(expert_off)
    _status(status)
    Mcap, K = xq.shape
    Mw, K_w = wq.shape
    if K_w != K:
        raise MgwError(f"wq [Mw, {K_w}] and xq [Mcap, {K}] must share the contraction width")
    _need(xs, K * Mcap // 32, "xs")
    _need(ws, K * Mw // 32, "ws")
    M, N, act = _size(M, "M"), _size(N, "N"), int(act)
    F = N // 2 if act in GATED_ACTS else N
    if bias is not None:
        _shaped(bias, (E, N), torch.float32, "bias")
    if residual is not None:
        _shaped(residual, (M, F), torch.bfloat16, "residual")
    dev = _one_device(xq, xs, wq, ws, expert_off, bias, residual, out, preact, status)
    side = None if stream is None else _side(stream, dev)
    out = _out(out, (M, F), torch.bfloat16, dev, "out", side)
    if save_preact or preact is not None:
        preact = _out(preact, (M, N), torch.bfloat16, dev, "preact", side)
    with _device(dev):
        st = load().mgw_grouped_fprop_mxfp8_act(
            _ptr(xq), _ptr(xs), _ptr(wq), _ptr(ws), _ptr(expert_off), E, M, N, K, Mcap, Mw, act,
            _ptr(bias), _ptr(residual), _ptr(out), _ptr(preact), _ptr(status), _stream(stream))
    _check(st, "mgw_grouped_fprop_mxfp8_act")
    if side is not None:
        _used_on(side, xq, xs, wq, ws, expert_off, bias, residual, out, preact, status)
    return out if preact is None else (out, preact)


def grouped_act_backward(dy: torch.Tensor, z: torch.Tensor | None, expert_off: torch.Tensor,
                         act: int, with_dbias: bool = False, dz: torch.Tensor | None = None,
                         dbias: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         status: torch.Tensor | None = None, stream=None):
    """-> (dz bf16 [M, N], dbias fp32 [E, N] or None): the backward pass of
    :func:`grouped_fprop_mxfp8_act`'s epilogue from dy [M, F] bf16 and the saved pre-activation
    z [M, N] bf16.  For ACT_NONE z is None and dz is dy itself.  ``workspace`` (uint8) is
    allocated when a large call with dbias needs one and none is given."""
    act = int(act)
    _dev_tensor(dy, torch.bfloat16, "dy", 2)
    M, F = dy.shape
    N = 2 * F if act in GATED_ACTS else F
    if act == ACT_NONE:
        if z is not None or dz is not None:
            raise MgwError("ACT_NONE takes no z and no dz: dz is dy")
    else:
        if z is None:
            raise MgwError("z (the saved pre-activation) is needed for this activation")
        _shaped(z, (M, N), torch.bfloat16, "z")
    E = _offsets(expert_off)
    _status(status)
    dev = _one_device(dy, z, expert_off, dz, dbias, workspace, status)
    side = None if stream is None else _side(stream, dev)
    if act != ACT_NONE:
        dz = _out(dz, (M, N), torch.bfloat16, dev, "dz", side)
    lib = load()
    if with_dbias or dbias is not None:
        dbias = _out(dbias, (E, N), torch.float32, dev, "dbias", side)
        need = int(lib.mgw_grouped_act_backward_workspace_bytes(E, M, N))
        if need or workspace is not None:
            workspace = _out(workspace, (need,), torch.uint8, dev, "workspace", side)
    with _device(dev):
        st = lib.mgw_grouped_act_backward(_ptr(dy), _ptr(z), _ptr(expert_off), E, M, N, act,
                                          _ptr(dz), _ptr(dbias), _ptr(workspace),
                                          0 if workspace is None else workspace.numel(),
                                          _ptr(status), _stream(stream))
    _check(st, "mgw_grouped_act_backward")
    if side is not None:
        _used_on(side, dy, z, expert_off, dz, dbias, workspace, status)
    return (dy if act == ACT_NONE else dz), dbias


def moe_combine(y: torch.Tensor, row_of: torch.Tensor, weights: torch.Tensor | None = None,
                residual: torch.Tensor | None = None, out: torch.Tensor | None = None,
                status: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out [T, H] = residual[t] + sum_k weights[t, k] * y[row_of[t, k]], y [M, H] bf16 or fp32,
    row_of int32 [T, top_k] (-1: dropped) from :func:`moe_dispatch`.  Without weights every
    weight is 1: the gradient of gathering the routed rows."""
    dt = _element_type(y, "y")
    _dev_tensor(y, y.dtype, "y", 2)
    M, H = y.shape
    _dev_tensor(row_of, torch.int32, "row_of", 2)
    T, top_k = row_of.shape
    if weights is not None:
        _shaped(weights, (T, top_k), torch.float32, "weights")
    if residual is not None:
        _shaped(residual, (T, H), y.dtype, "residual")
    _status(status)
    dev = _one_device(y, row_of, weights, residual, out, status)
    side = None if stream is None else _side(stream, dev)
    out = _out(out, (T, H), y.dtype, dev, "out", side)
    with _device(dev):
        st = load().mgw_moe_combine(_ptr(y), dt, M, _ptr(row_of), _ptr(weights), _ptr(residual), T,
                                    top_k, H, _ptr(out), _ptr(status), _stream(stream))
    _check(st, "mgw_moe_combine")
    if side is not None:
        _used_on(side, y, row_of, weights, residual, out, status)
    return out


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor | None, row_of: torch.Tensor,
                         weights: torch.Tensor | None = None, M: int | None = None,
                         dy: torch.Tensor | None = None, dweights: torch.Tensor | None = None,
                         status: torch.Tensor | None = None, stream=None):
    """-> (dy [M, H], dweights fp32 [T, top_k] or None): the backward pass of
    :func:`moe_combine`.  Without weights there is no dweights, y may be None and M is given
    instead.  Rows of dy that no pair of ``row_of`` names are not written."""
    dt = _element_type(dout, "dout")
    _dev_tensor(dout, dout.dtype, "dout", 2)
    T, H = dout.shape
    _dev_tensor(row_of, torch.int32, "row_of", 2)
    top_k = row_of.shape[1]
    _shaped(row_of, (T, top_k), torch.int32, "row_of")
    if weights is not None:
        _shaped(weights, (T, top_k), torch.float32, "weights")
        if y is None:
            raise MgwError("y is needed for the gradient of the weights")
    elif dweights is not None:
        raise MgwError("dweights needs weights")
    if y is not None:
        _dev_tensor(y, dout.dtype, "y", 2)
        if y.shape[1] != H or (M is not None and y.shape[0] != int(M)):
            raise MgwError(f"y {tuple(y.shape)} does not match dout [T, {H}] or M")
        M = y.shape[0]
    elif M is None:
        raise MgwError("M (the number of routed rows) is needed without y")
    M = _size(M, "M")
    _status(status)
    dev = _one_device(dout, y, row_of, weights, dy, dweights, status)
    side = None if stream is None else _side(stream, dev)
    dy = _out(dy, (M, H), dout.dtype, dev, "dy", side)
    if weights is not None:
        dweights = _out(dweights, (T, top_k), torch.float32, dev, "dweights", side)
    with _device(dev):
        st = load().mgw_moe_combine_backward(_ptr(dout), _ptr(y), dt, M, _ptr(row_of),
                                             _ptr(weights), T, top_k, H, _ptr(dy), _ptr(dweights),
                                             _ptr(status), _stream(stream))
    _check(st, "mgw_moe_combine_backward")
    if side is not None:
        _used_on(side, dout, y, row_of, weights, dy, dweights, status)
    return dy, dweights


# ------------------------------------------------------------- operators in modules of their own
_ELSEWHERE = {"grouped_lora": "adapters", "grouped_lora_backward": "adapters",
              "GradTable": "gradients", "grad_norm": "gradients", "clip_grads": "gradients"}
_found = {}


def __getattr__(name):
    """``mgw.grouped_lora`` and the others of :mod:`.adapters` and :mod:`.gradients`, which build on
    this module."""
    f = _found.get(name)
    if f is None:
        module = _ELSEWHERE.get(name)
        if module is None:
            raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
        f = _found[name] = getattr(importlib.import_module("." + module, __package__), name)
    return f
