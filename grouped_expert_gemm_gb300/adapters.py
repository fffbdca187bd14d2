"""Low-rank adapters beside a shared projection, and gradient clipping, on the library's calls.

``AdapterProjection``  y = x W + scale (x A^T) B for a batch whose segments of rows each have an
                       adapter of their own or none: a serving step of many requests, or a
                       training step of several adapters side by side, with its backward.
                       With ``y_dtype=torch.float32`` y can be the router's logits.
``GradientClip``       the gradient norm over many tensors, or one for each group of them (one
                       adapter's, say), and the tensors scaled to a largest norm.

As the layers: each object owns its buffers, a call only enqueues kernels on the given stream
(default: the current one) and can be captured into a CUDA graph; arguments are checked with
ValueError, and the object's device must be the current one.  Calls of one object share its
buffers: they follow one another on the GPU.  An object is made outside of captures.
"""
from __future__ import annotations

import math
from typing import Optional, Sequence

import torch

from . import abi
from .block import _KIND, _device, check_tensor


def _not_capturing(device):
    if device.type == "cuda" and torch.cuda.is_current_stream_capturing():
        raise ValueError("the object must be made before a capture begins")


def _check_rows(name, t, shape, dtype, device):
    """As check_tensor with rows at any distance that is a multiple of 8 values."""
    check_tensor(name, t, shape, dtype, device, rows_strided=True)
    if shape[0] > 1 and t.stride(0) % 8 != 0:
        raise ValueError(f"rows of {name} must be a multiple of 8 values apart")


def _overlap(p, q) -> bool:
    """Whether two tensors with contiguous rows share memory.  Slices of the columns of one wider
    buffer may stand side by side in its rows."""
    if p.numel() == 0 or q.numel() == 0:
        return False
    at, size = [], []
    for t in (p, q):
        at.append(t.data_ptr())
        rows = t.dim() == 2 and t.shape[0] > 1
        values = (t.shape[0] - 1) * t.stride(0) + t.shape[1] if rows else t.numel()
        size.append(values * t.element_size())
    if at[0] + size[0] <= at[1] or at[1] + size[1] <= at[0]:
        return False
    if p.dim() == q.dim() == 2 and min(p.shape[0], q.shape[0]) > 1:
        # every row of either starts at its place in a row of this many bytes
        row = math.gcd(p.stride(0) * p.element_size(), q.stride(0) * q.element_size())
        ahead = (at[1] - at[0]) % row
        return ahead < p.shape[1] * p.element_size() or \
            ahead + q.shape[1] * q.element_size() > row
    return True


def _apart(name, written, *read):
    """What a call writes must not be what other blocks of it still read."""
    for t in read:
        if t is not None and _overlap(written, t):
            raise ValueError(f"{name} must not overlap what the call reads")


def _stride(t, width):
    return t.stride(0) if t.shape[0] > 1 else width


class AdapterProjection:
    """weight [d, n] bf16 (frozen), tables a [N, r, d] and b [N, r, n] bf16 and scale [N] fp32:
    the adapters, which the caller may change in place between steps.

    ``forward(x, seg_adapter, seg_offsets)``: segment q holds rows [seg_offsets[q],
    seg_offsets[q+1]) of x [T, d] and has adapter seg_adapter[q] (-1: none); int32 tensors
    [n_seg] and [n_seg + 1] (None: one segment of all rows).  Returns y [T, n]; rows of no
    segment keep what they held (zeros at first).  ``u`` [T, r] is what the backward needs.

    ``gradients``: make the backward's buffers (dx, da, db and a workspace) too; a program that
    serves alone can do without them.  They are made here and not by the first backward: one that is
    captured would clear them in every replay."""

    def __init__(self, T: int, weight: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
                 scale: torch.Tensor, y_dtype=torch.bfloat16, device="cuda",
                 gradients: bool = True):
        self.device = _device(device)
        _not_capturing(self.device)
        if y_dtype not in _KIND:
            raise ValueError("y_dtype must be bfloat16 or float32")
        for name, t, dims in (("weight", weight, 2), ("a", a, 3), ("b", b, 3)):
            if not isinstance(t, torch.Tensor) or t.dim() != dims:
                raise ValueError(f"{name} must be a tensor of {dims} dimensions")
        self.T, (self.d, self.n), (self.N, self.r) = T, weight.shape, a.shape[:2]
        check_tensor("weight", weight, (self.d, self.n), torch.bfloat16, self.device)
        check_tensor("a", a, (self.N, self.r, self.d), torch.bfloat16, self.device)
        check_tensor("b", b, (self.N, self.r, self.n), torch.bfloat16, self.device)
        check_tensor("scale", scale, (self.N,), torch.float32, self.device)
        self.weight, self.a, self.b, self.scale, self.y_dtype = weight, a, b, scale, y_dtype
        self.params = abi.AdapterParams(T, self.d, self.n, self.r, self.N, 1, _KIND[y_dtype])
        self.ws_bytes = abi.moe_adapter_project_backward_workspace_size(self.params)
        if self.ws_bytes == 0:
            raise ValueError("unsupported shape (d, n and r multiples of 8, d, n <= 65536, "
                             "r <= 128, at most 65535 adapters)")
        new = dict(device=self.device)
        self.u = torch.zeros((T, self.r), dtype=torch.float32, **new)
        self.y = torch.zeros((T, self.n), dtype=y_dtype, **new)
        self.dev_status = torch.zeros((1,), dtype=torch.int32, **new)
        self._last = None
        self._grads = None if not gradients else (
            torch.zeros((T, self.d), dtype=torch.bfloat16, **new),
            torch.zeros(a.shape, dtype=torch.float32, **new),
            torch.zeros(b.shape, dtype=torch.float32, **new),
            torch.empty((self.ws_bytes,), dtype=torch.uint8, **new))
        if self.device.type == "cuda":  # the buffers are clear whatever stream uses them
            torch.cuda.current_stream(self.device).synchronize()

    def _segments(self, seg_adapter, seg_offsets):
        n_seg = seg_adapter.shape[0] if isinstance(seg_adapter, torch.Tensor) and \
            seg_adapter.dim() == 1 else 0
        if not 1 <= n_seg <= 65535:
            raise ValueError("seg_adapter must hold one id for each of 1 to 65535 segments")
        check_tensor("seg_adapter", seg_adapter, (n_seg,), torch.int32, self.device)
        if seg_offsets is not None:
            check_tensor("seg_offsets", seg_offsets, (n_seg + 1,), torch.int32, self.device)
        elif n_seg != 1:
            raise ValueError("several segments need seg_offsets")
        return n_seg

    def forward(self, x, seg_adapter, seg_offsets=None, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
        """``out``: write there instead of ``y`` (rows at any multiple of 8 values apart, a
        slice of a wider buffer for example).  Neither may overlap what the call reads."""
        abi.check_current_device(self.device)
        _check_rows("x", x, (self.T, self.d), torch.bfloat16, self.device)
        p = self.params
        n_seg = self._segments(seg_adapter, seg_offsets)
        y = self.y if out is None else out
        if out is not None:
            _check_rows("out", out, (self.T, self.n), self.y_dtype, self.device)
            _apart("out", out, self.weight, self.a, self.b, self.scale, self.u, seg_adapter,
                   seg_offsets)
        _apart("y", y, x)
        p.n_seg, p.x_stride, p.y_stride = n_seg, _stride(x, self.d), _stride(y, self.n)
        abi.moe_adapter_project(p, seg_offsets, seg_adapter, x, self.weight, self.a, self.b,
                                self.scale, self.u, y, self.dev_status, stream)
        self._last = (x, seg_adapter, seg_offsets)
        return y

    def backward(self, dy, accumulate: bool = False, stream=None):
        """Gradients of the last forward, whose x, segments and tables must be as they were:
        (dx [T, d] bf16, da, db fp32 like the tables); dy is [T, n] bf16.  The buffers are the
        object's own; with ``accumulate`` da and db are added to what they hold (zeros at first),
        in a captured call by every replay.  The weight has no gradient."""
        abi.check_current_device(self.device)
        if self._grads is None:
            raise ValueError("the object was made without gradients")
        if self._last is None:
            raise ValueError("backward needs a forward before it")
        _check_rows("dy", dy, (self.T, self.n), torch.bfloat16, self.device)
        x, seg_adapter, seg_offsets = self._last
        _apart("dx", self._grads[0], dy, x)
        dx, da, db, ws = self._grads
        p = self.params
        p.n_seg = self._segments(seg_adapter, seg_offsets)
        p.x_stride, p.y_stride = _stride(x, self.d), _stride(dy, self.n)
        abi.moe_adapter_project_backward(p, seg_offsets, seg_adapter, x, self.weight, self.a,
                                         self.b, self.scale, self.u, dy, dx, da, db,
                                         int(accumulate), ws, self.ws_bytes, self.dev_status,
                                         stream)
        return dx, da, db


class GradientClip:
    """Scales gradients so that the norm of each group of them is at most max_norm.

    grads: bf16 and fp32 tensors (contiguous; tensors that overlap are refused).  max_norm:
    infinity scales nothing, whatever the norm.  out: where the scaled ones go, like grads
    (default: in place).  groups: the group of each (default: one group of all); n_groups: how
    many there are.  ``clip()`` returns ``norms`` [n_groups], the norms before scaling.  The table
    of the tensors is made once, here, and names their memory: the tensors are kept alive, and a
    program that replaces one makes another object."""

    def __init__(self, grads: Sequence[torch.Tensor], max_norm: float, out=None, groups=None,
                 n_groups: Optional[int] = None, norms: Optional[torch.Tensor] = None,
                 device="cuda"):
        self.device = _device(device)
        _not_capturing(self.device)
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        groups = [0] * len(self.grads) if groups is None else [int(g) for g in groups]
        if len(self.out) != len(self.grads) or len(groups) != len(self.grads):
            raise ValueError("out and groups must have one entry for each gradient")
        self.n_groups = (max(groups) + 1 if groups else 1) if n_groups is None else n_groups
        if not 1 <= self.n_groups <= 1 << 20 or any(not 0 <= g < self.n_groups for g in groups):
            raise ValueError("groups must be in [0, n_groups), n_groups in [1, 2^20]")
        if not max_norm > 0:
            raise ValueError("max_norm must be positive")
        self.max_norm = float(max_norm)
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            if not isinstance(g, torch.Tensor) or g.dtype not in _KIND:
                raise ValueError(f"grads[{i}] must be a bfloat16 or float32 tensor")
            check_tensor(f"grads[{i}]", g, g.shape, g.dtype, self.device)
            check_tensor(f"out[{i}]", o, g.shape, g.dtype, self.device)
        # Each tensor's bytes once (in place: gradient and result are the same ones): elements that
        # two blocks read and write would be scaled in any order, or twice.
        spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
                       for g, o in zip(self.grads, self.out)
                       for t in ((g,) if g.data_ptr() == o.data_ptr() else (g, o)) if t.numel())
        if any(end > begin for (_, end), (begin, _) in zip(spans, spans[1:])):
            raise ValueError("gradients and their results must not overlap")
        table = (abi.GradTensor * len(self.grads))()
        for t, i in zip(table, sorted(range(len(self.grads)), key=lambda i: groups[i])):
            g, o = self.grads[i], self.out[i]
            t.grad, t.out, t.count = g.data_ptr() or None, o.data_ptr() or None, g.numel()
            t.type, t.group = _KIND[g.dtype], groups[i]
        self.n_chunks = abi.moe_grad_plan(table, self.n_groups)
        new = dict(device=self.device)
        self.norms = torch.zeros((self.n_groups,), dtype=torch.float32, **new) \
            if norms is None else norms
        check_tensor("norms", self.norms, (self.n_groups,), torch.float32, self.device)
        first = self.norms.data_ptr()
        if any(first < end and begin < first + 4 * self.n_groups for begin, end in spans):
            raise ValueError("norms must not overlap a gradient or its result")
        host = torch.frombuffer(bytearray(bytes(table)) or bytearray(8), dtype=torch.uint8)
        self.table = host.to(self.device)
        self.ws_bytes = abi.moe_clip_grads_workspace_size(self.n_groups)
        self.ws = torch.empty((self.ws_bytes,), dtype=torch.uint8, **new)
        self.dev_status = torch.zeros((1,), dtype=torch.int32, **new)
        if self.device.type == "cuda":  # the table is there whatever stream uses it
            torch.cuda.current_stream(self.device).synchronize()

    def clip(self, stream=None) -> torch.Tensor:
        abi.check_current_device(self.device)
        abi.moe_clip_grads(len(self.grads), self.table, self.n_chunks, self.n_groups,
                           self.max_norm, self.norms, self.ws, self.ws_bytes, self.dev_status,
                           stream)
        return self.norms
