"""Low-rank adapters of many requests at once beside a shared projection, forward and backward:
the binding of mgw_grouped_lora and mgw_grouped_lora_backward (include/mgw.h).

Rows are sorted by adapter, as the grouped products' are by expert; :func:`mgw.moe_dispatch` makes
their tables.  Also reached as ``mgw.grouped_lora`` and ``mgw.grouped_lora_backward``; checks, streams
and errors are :mod:`mgw`'s.
"""
from __future__ import annotations

import torch

from . import mgw


def _adapters(a, b, adapter_off, scale, row_index, out_index):
    """Checks the adapters and the row tables; returns (E, R, K, N)."""
    mgw._dev_tensor(a, torch.bfloat16, "a", 3)
    E, R, K = a.shape
    mgw._dev_tensor(b, torch.bfloat16, "b", 3)
    N = b.shape[1]
    mgw._shaped(b, (E, N, R), torch.bfloat16, "b")
    mgw._dev_tensor(adapter_off, torch.int32, "adapter_off", 1)
    if adapter_off.numel() != E + 1:
        raise mgw.MgwError(f"adapter_off has {adapter_off.numel()} entries; {E} adapters need {E + 1}")
    if scale is not None:
        mgw._shaped(scale, (E,), torch.float32, "scale")
    if row_index is not None:
        mgw._dev_tensor(row_index, torch.int32, "row_index", 1)
    if out_index is not None:
        mgw._dev_tensor(out_index, torch.int32, "out_index", 1)
        if row_index is not None and row_index.numel() != out_index.numel():
            raise mgw.MgwError(f"row_index and out_index name {row_index.numel()} and {out_index.numel()} rows")
    return E, R, K, N


def _adapter_rows(x_rows: int, rows: int | None, row_index, out_index, of: str) -> tuple[int, int]:
    """(M, the rows of ``of``): as many rows as an index names, or as x has; ``rows`` None: M."""
    index = row_index if row_index is not None else out_index
    M = x_rows if index is None else index.numel()
    rows = M if rows is None else rows
    if (row_index is None and x_rows < M) or (out_index is None and rows < M):
        raise mgw.MgwError(f"{M} rows need an index, or as many rows of x ({x_rows}) and of {of} ({rows})")
    if max(x_rows, rows, M) > mgw.MAX_SIZE:
        raise mgw.MgwError("a number of rows exceeds the C ABI's 32-bit sizes")
    return M, rows


_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _fit(x, a, b, adapter_off, row_index, out_index, scale, out_like, u=None, x_like=None) -> bool:
    """The usual call's check in one pass (5 us less than one by one): every tensor has its type, shape
    and the device of x, and is contiguous.  ``out_like`` has out's columns, ``x_like`` x's and the rows
    of out_like.  Whoever gets False goes through the single checks, which say what is wrong."""
    try:
        d = x.get_device()
        E, R, K = a.size()
        N = b.size(1)
        index = row_index if row_index is not None else out_index
        M = x.size(0) if index is None else index.size(0)
        return (d >= 0 and a.get_device() == b.get_device() == adapter_off.get_device() == d
                and x.dtype is _BF16 and a.dtype is _BF16 and b.dtype is _BF16 and adapter_off.dtype is _I32
                and x.size() == (x.size(0), K) and b.size() == (E, N, R) and adapter_off.size() == (E + 1,)
                and x.is_contiguous() and a.is_contiguous() and b.is_contiguous() and adapter_off.is_contiguous()
                and (row_index is None or row_index.get_device() == d and row_index.dtype is _I32
                     and row_index.size() == (M,) and row_index.is_contiguous())
                and (out_index is None or out_index is row_index or out_index.get_device() == d
                     and out_index.dtype is _I32 and out_index.size() == (M,) and out_index.is_contiguous())
                and (scale is None or scale.get_device() == d and scale.dtype is _F32 and scale.size() == (E,)
                     and scale.is_contiguous())
                and (out_like is None or out_like.get_device() == d and out_like.dtype is _BF16
                     and out_like.size() == (out_like.size(0), N) and out_like.is_contiguous())
                and (u is None or u.get_device() == d and u.dtype is _F32 and u.size() == (M, R)
                     and u.is_contiguous())
                and (x_like is None or x_like.get_device() == d and x_like.dtype is _BF16
                     and x_like.size() == (out_like.size(0), K) and x_like.is_contiguous()))
    except (AttributeError, IndexError, TypeError, ValueError):
        return False


def grouped_lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, adapter_off: torch.Tensor,
                 row_index: torch.Tensor | None = None, out_index: torch.Tensor | None = None,
                 scale: torch.Tensor | None = None, base: torch.Tensor | None = None,
                 save_u: bool = False, out: torch.Tensor | None = None, u: torch.Tensor | None = None,
                 status: torch.Tensor | None = None, stream=None):
    """out[o] = base[o] + scale[e] * (x[t] a[e]^T) b[e]^T for every row of every adapter, x [rows, K]
    bf16, a [E, R, K], b [E, N, R] -> out [rows of base, N] bf16; with ``save_u`` (or ``u``) also the
    intermediate u = x a^T, fp32 [M, R], for :func:`grouped_lora_backward`.

    Adapter e has the rows adapter_off[e] .. adapter_off[e+1]-1; row r reads x[row_index[r]] and is
    out's row out_index[r] (r itself without an index).  Rows behind adapter_off[E] have no adapter
    and keep their base.  For requests in token order both indices are the row_index of
    :func:`moe_dispatch` (top_k 1; an extra last expert for tokens without an adapter, whose offset
    is left out of ``adapter_off``).  ``base`` is 0 when not given, and may be ``out``, as may x (of
    as many columns) where no row reads a row of x that another writes; other overlaps of outputs and
    inputs are refused.  Rows of out that ``out_index`` does not name are not written."""
    fit = _fit(x, a, b, adapter_off, row_index, out_index, scale, base)
    if not fit:
        mgw._dev_tensor(x, torch.bfloat16, "x", 2)
        K = _adapters(a, b, adapter_off, scale, row_index, out_index)[2]
        if x.shape[1] != K:
            raise mgw.MgwError(f"x [rows, {x.shape[1]}] and a [E, R, {K}] must share the contraction width")
        if base is not None:
            mgw._dev_tensor(base, torch.bfloat16, "base", 2)
            mgw._shaped(base, (base.shape[0], b.shape[1]), torch.bfloat16, "base")
    E, R, K = a.shape
    N = b.shape[1]
    rows = None
    if base is not None:
        rows = base.shape[0]
    elif isinstance(out, torch.Tensor) and out.dim() == 2:
        rows = out.shape[0]
    M, rows = _adapter_rows(x.shape[0], rows, row_index, out_index, "out")
    mgw._status(status)
    dev = mgw._one_device(x, out, u, status) if fit else \
        mgw._one_device(x, a, b, adapter_off, row_index, out_index, scale, base, out, u, status)
    side = None if stream is None else mgw._side(stream, dev)
    out = mgw._out(out, (rows, N), torch.bfloat16, dev, "out", side)
    if save_u or u is not None:
        u = mgw._out(u, (M, R), torch.float32, dev, "u", side)
    with mgw._device(dev):
        st = mgw.load().mgw_grouped_lora(x.data_ptr(), x.shape[0], mgw._ptr(row_index), M, K, a.data_ptr(),
                                     b.data_ptr(), mgw._ptr(scale), adapter_off.data_ptr(), E, R, N,
                                     mgw._ptr(base), mgw._ptr(out_index), rows, out.data_ptr(), mgw._ptr(u),
                                     mgw._ptr(status), mgw._stream(stream))
    if st:
        mgw._check(st, "mgw_grouped_lora")
    if side is not None:
        mgw._used_on(side, x, a, b, adapter_off, row_index, out_index, scale, base, out, u, status)
    return out if u is None else (out, u)


def grouped_lora_backward(dy: torch.Tensor, x: torch.Tensor | None, u: torch.Tensor | None,
                          a: torch.Tensor, b: torch.Tensor, adapter_off: torch.Tensor,
                          row_index: torch.Tensor | None = None, out_index: torch.Tensor | None = None,
                          scale: torch.Tensor | None = None, dx_base: torch.Tensor | None = None,
                          with_dx: bool = True, with_weights: bool = True,
                          dx: torch.Tensor | None = None, da: torch.Tensor | None = None,
                          db: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, stream=None):
    """-> (dx, da, db): the backward pass of :func:`grouped_lora` from dy [rows of out, N] bf16.
    dx [rows of out, K] bf16 = dx_base + the adapters' share (rows without an adapter: dx_base, 0
    when not given; ``dx_base`` may be ``dx``), da [E, R, K] and db [E, N, R] bf16; ``x`` and ``u``
    as in the forward call.  Without ``with_dx`` dx is None; without ``with_weights`` da and db are,
    and ``x`` and ``u`` may be None, and ``dx`` may be dy (of as many columns).  Other overlaps of
    outputs and inputs are refused.  ``workspace`` (uint8) is allocated when none is given."""
    if not with_dx and (dx is not None or dx_base is not None):
        raise mgw.MgwError("dx and dx_base need with_dx")
    if not with_weights and (da is not None or db is not None):
        raise mgw.MgwError("da and db need with_weights")
    if with_weights and (x is None or u is None):
        raise mgw.MgwError("x and u are needed for the adapters' gradients")
    if not with_weights:
        x = u = None
    fit = with_weights and _fit(x, a, b, adapter_off, row_index, out_index, scale, dy, u, dx_base)
    if not fit:
        mgw._dev_tensor(dy, torch.bfloat16, "dy", 2)
        _, _, K, N = _adapters(a, b, adapter_off, scale, row_index, out_index)
        if dy.shape[1] != N:
            raise mgw.MgwError(f"dy [rows, {dy.shape[1]}] does not match b [E, {N}, R]")
        if x is not None:
            mgw._dev_tensor(x, torch.bfloat16, "x", 2)
            if x.shape[1] != K:
                raise mgw.MgwError(f"x [rows, {x.shape[1]}] and a [E, R, {K}] must share the contraction width")
    E, R, K = a.shape
    N = b.shape[1]
    x_rows = dy.shape[0] if x is None else x.shape[0]
    M, rows = _adapter_rows(x_rows, dy.shape[0], row_index, out_index, "dy")
    if not fit and u is not None:
        mgw._shaped(u, (M, R), torch.float32, "u")
    if not fit and dx_base is not None:
        mgw._shaped(dx_base, (rows, K), torch.bfloat16, "dx_base")
    mgw._status(status)
    dev = mgw._one_device(dy, dx, da, db, workspace, status) if fit else \
        mgw._one_device(dy, x, u, a, b, adapter_off, row_index, out_index, scale, dx_base, dx, da, db,
                    workspace, status)
    side = None if stream is None else mgw._side(stream, dev)
    lib = mgw.load()
    if with_dx:
        dx = mgw._out(dx, (rows, K), torch.bfloat16, dev, "dx", side)
    if with_weights:
        da = mgw._out(da, (E, R, K), torch.bfloat16, dev, "da", side)
        db = mgw._out(db, (E, N, R), torch.bfloat16, dev, "db", side)
        need = int(lib.mgw_grouped_lora_backward_workspace_bytes(E, M, K, N, R))
        workspace = mgw._out(workspace, (need,), torch.uint8, dev, "workspace", side)
    with mgw._device(dev):
        st = lib.mgw_grouped_lora_backward(dy.data_ptr(), rows, mgw._ptr(out_index), mgw._ptr(x), x_rows,
                                           mgw._ptr(row_index), M, K, a.data_ptr(), b.data_ptr(),
                                           mgw._ptr(scale), adapter_off.data_ptr(), E, R, N, mgw._ptr(u),
                                           mgw._ptr(dx_base), mgw._ptr(dx), mgw._ptr(da), mgw._ptr(db),
                                           mgw._ptr(workspace), 0 if workspace is None else workspace.numel(),
                                           mgw._ptr(status), mgw._stream(stream))
    if st:
        mgw._check(st, "mgw_grouped_lora_backward")
    if side is not None:
        mgw._used_on(side, dy, x, u, a, b, adapter_off, row_index, out_index, scale, dx_base, dx, da, db,
                 workspace, status)
    return dx, da, db
