"""The norm of all gradients of a model together, and the gradients clipped to a largest norm: the
binding of mgw_grad_norm and mgw_grad_clip (include/mgw.h).

Also reached as ``mgw.GradTable``, ``mgw.grad_norm`` and ``mgw.clip_grads``; checks, streams and errors
are :mod:`mgw`'s.
"""
from __future__ import annotations

import bisect
import ctypes
import operator

import torch

from . import mgw

_SHIFT = {mgw.TYPE_BF16: 1, mgw.TYPE_F32: 2}  # an element's bytes


class GradTable:
    """The gradients (bf16 and fp32 tensors, any sizes, contiguous, on one device) that
    :func:`grad_norm` and :func:`clip_grads` take, checked once: for a program whose gradient buffers
    stay where they are from step to step, and for captured calls.  ``out``: tensors of the same
    types and sizes that the clipped gradients go to, the gradients themselves or memory that
    overlaps none of the call's tensors (without it: in place; clipping refuses other overlaps).
    Holds the tensors; one whose memory is replaced afterwards (``t.data = ..``, ``resize_``) needs a
    new table."""

    def __init__(self, grads, out=None):
        self.grads = list(grads)
        self.out = None if out is None else list(out)
        self.device, self._kinds, sizes = self._checked(self.grads, "grads")
        n = self.n = len(self.grads)
        at = grads_at = [t.data_ptr() for t in self.grads]
        self._grads = (ctypes.c_void_p * n)(*at)
        self._sizes = (ctypes.c_int64 * n)(*sizes)
        self._dtypes = (ctypes.c_int * n)(*self._kinds)
        self._out = None
        if self.out is not None:
            dev, kinds, out_sizes = self._checked(self.out, "out")
            if kinds != self._kinds or out_sizes != sizes or (n and dev != self.device):
                raise mgw.MgwError("out must hold one tensor of the same type, size and device for every gradient")
            at = [t.data_ptr() for t in self.out]
            self._out = (ctypes.c_void_p * n)(*at)
        self._workspace = int(mgw.load().mgw_grad_workspace_bytes(mgw._size(n, "the number of gradients")))
        # where the gradients and the outputs lie, for the first clipping
        self._places = (grads_at, at, sizes)
        self._overlap = None

    def _overlaps(self) -> bool:
        """Whether memory that clipping writes meets another tensor of the table: looked for once, at the
        first clipping."""
        if self._overlap is None:
            at, to, sizes = self._places
            # Spans are apart where each ends, in order, before the next begins.  (Sorted without their
            # owners: 128 gradients of a list take 10 us so, 40 as a sweep over pairs.)
            starts = sorted(to if all(sizes) else [p for p, n in zip(to, sizes) if n])
            ends = sorted([p + (n << _SHIFT[k]) for p, n, k in zip(to, sizes, self._kinds) if n])
            overlap = not all(map(operator.le, ends, starts[1:]))
            if not overlap and at is not to:
                # no gradient but an output's own lies on an output
                overlap = any(n and p != q and bisect.bisect_right(ends, p) != bisect.bisect_left(starts, p + (n << _SHIFT[k]))
                              for p, q, n, k in zip(at, to, sizes, self._kinds))
            self._overlap = overlap
        return self._overlap

    @staticmethod
    def _checked(ts, name):
        dev, kinds, sizes = None, [], []
        for t in ts:
            kinds.append(mgw._element_type(t, name))
            if not mgw._on_cuda(t):
                raise mgw.MgwError(f"{name} must be CUDA tensors")
            if not t.is_contiguous():
                raise mgw.MgwError(f"{name} must be contiguous")
            if dev is None:
                dev = t.device
            elif t.device != dev:
                raise mgw.MgwError(f"all tensors must be on one CUDA device, got {dev} and {t.device} in {name}")
            sizes.append(t.numel())
        return dev, kinds, sizes


def _grad_call(grads, norm, workspace, stream):
    """The table of ``grads`` and the checked or new workspace -> (table, device, side, workspace)."""
    table = grads if isinstance(grads, GradTable) else GradTable(grads)
    dev = table.device
    if dev is None:  # no gradients at all
        dev = torch.device("cuda", torch.cuda.current_device())
    if norm is not None:
        mgw._dev_tensor(norm, torch.float32, "norm")
        mgw._need(norm, 1, "norm")
    if workspace is not None:
        mgw._dev_tensor(workspace, torch.uint8, "workspace")
    for t in (norm, workspace):
        if t is not None and t.device != dev:
            raise mgw.MgwError(f"all tensors must be on one CUDA device, got {sorted({str(dev), str(t.device)})}")
    side = None if stream is None else mgw._side(stream, dev)
    workspace = mgw._out(workspace, (table._workspace,), torch.uint8, dev, "workspace", side)
    return table, dev, side, workspace


def grad_norm(grads, norm: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """The norm of all ``grads`` together (a :class:`GradTable` or a list of bf16 and fp32 tensors)
    -> fp32 [1]: sqrt of the sum of all elements' squares, 0 for no elements."""
    table, dev, side, workspace = _grad_call(grads, norm, workspace, stream)
    norm = mgw._out(norm, (1,), torch.float32, dev, "norm", side)
    with mgw._device(dev):
        st = mgw.load().mgw_grad_norm(table._grads, table._sizes, table._dtypes, table.n, mgw._ptr(norm),
                                  mgw._ptr(workspace), workspace.numel(), mgw._stream(stream))
    mgw._check(st, "mgw_grad_norm")
    if side is not None:
        mgw._used_on(side, norm, workspace, *table.grads)
    return norm


def clip_grads(grads, max_norm: float, norm: torch.Tensor | None = None, known_norm: torch.Tensor | None = None,
               eps: float = 1e-6, workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Multiplies all ``grads`` (a :class:`GradTable`, into its ``out`` if it has one, or a list) by
    min(1, max_norm / (norm + eps)) -> their norm, fp32 [1], as :func:`grad_norm` gives it.
    ``known_norm`` (fp32 [1]), where given, is taken for the norm and returned: that of several
    processes' gradients, for example."""
    table, dev, side, workspace = _grad_call(grads, norm, workspace, stream)
    if table._overlaps():
        raise mgw.MgwError("memory that is written belongs to two tensors of the call")
    if known_norm is not None:
        if norm is not None:
            raise mgw.MgwError("norm is not computed where known_norm is given")
        mgw._dev_tensor(known_norm, torch.float32, "known_norm")
        mgw._need(known_norm, 1, "known_norm")
        if known_norm.device != dev:
            raise mgw.MgwError(f"all tensors must be on one CUDA device, got {dev} and {known_norm.device}")
    else:
        norm = mgw._out(norm, (1,), torch.float32, dev, "norm", side)
    with mgw._device(dev):
        st = mgw.load().mgw_grad_clip(table._grads, table._out, table._sizes, table._dtypes, table.n,
                                  float(max_norm), float(eps), mgw._ptr(known_norm), mgw._ptr(norm),
                                  mgw._ptr(workspace), workspace.numel(), mgw._stream(stream))
    mgw._check(st, "mgw_grad_clip")
    if side is not None:
        mgw._used_on(side, norm, known_norm, workspace, *table.grads, *(table.out or ()))
    return norm if known_norm is None else known_norm
