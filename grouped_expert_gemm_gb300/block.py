"""What surrounds the MoE layer in a transformer block, on the library's calls.

``TokenNorm``   residual addition and RMS norm whose outputs are the layer's inputs: bf16
                token rows for the router (and bf16 experts) and/or the E4M3 dispatch payload
                for ``MoELayer(payload="fp8_...")``; with its backward.
``RouterLoss``  the router's balance loss with per-expert counts over ragged sequences, and
                the logits' gradient (the loss's and the gates').
``quantize_weights``  bf16 expert weights to the E4M3 form ``MoELayer`` takes.

Like the layers, each object owns its buffers (allocated once) and a call only enqueues
kernels on the given stream (default: the current one), so calls can be captured into a CUDA
graph.  Arguments are checked here (type, shape, device, contiguity) with ValueError; the
object's device must be the current one.
"""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import abi
from .layer import PAYLOADS

_KIND = {torch.bfloat16: abi.MOE_DTYPE_BF16, torch.float32: abi.MOE_DTYPE_FP32}


def check_tensor(name: str, t, shape, dtype, device, rows_strided: bool = False):
    """A device tensor of exactly this shape and type, contiguous (or, with rows_strided,
    with contiguous rows at any distance)."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}, got {t.dtype} "
                         f"{tuple(t.shape)}")
    if not t.is_contiguous():
        if not (rows_strided and t.dim() == 2 and t.stride(1) == 1 and
                t.stride(0) >= t.shape[1]):
            raise ValueError(f"{name} must be contiguous")


def _device(device) -> torch.device:
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        return torch.device("cuda", torch.cuda.current_device())
    return d


def _memory_of(stream, device):
    """Where a call allocates: new memory belongs to the stream that the call runs on, since
    the current stream's may still be in use by work queued there."""
    if stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    return torch.cuda.stream(stream)


def quantize_weights(w: torch.Tensor, dev_status=None, stream=None):
    """Expert weights bf16 [E, K, N] (the layout of the bf16 passes) to (codes [E, N, K]
    float8_e4m3fn, scales fp32 [E, ceil(N/128), ceil(K/128)]), allocated on the call's stream;
    done once per set of weights."""
    if not (isinstance(w, torch.Tensor) and w.is_cuda and w.dtype == torch.bfloat16 and
            w.dim() == 3 and w.is_contiguous()):
        raise ValueError("weights must be a contiguous bf16 device tensor [E, K, N]")
    abi.check_current_device(w.device)
    E, K, N = w.shape
    with _memory_of(stream, w.device):
        q = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=w.device)
        s = torch.empty((E, -(-N // 128), -(-K // 128)), dtype=torch.float32, device=w.device)
    abi.moe_quantize_weights_fp8(E, K, N, w, q, s, dev_status, stream)
    return q, s


class TokenNorm:
    """h = round(x + residual); y = h / rms(h) * weight, as bf16 rows and/or E4M3 codes.

    ``payload``: "bf16" (y only), "fp8_row" or "fp8_block128" (codes ``xq`` and scales ``xs``,
    and with ``keep_bf16`` y as well, for the router).  x is [n, d] (x_dtype, rows at any
    multiple of 8 values apart), residual [n, d] (residual_dtype) or None (then h = x)."""

    def __init__(self, n: int, d: int, weight: torch.Tensor, eps: float = 1e-6,
                 x_dtype=torch.bfloat16, residual_dtype: Optional[torch.dtype] = torch.bfloat16,
                 payload: str = "bf16", keep_bf16: bool = True, device="cuda"):
        if payload not in PAYLOADS:
            raise ValueError(f"payload must be one of {sorted(PAYLOADS)}")
        if x_dtype not in _KIND or residual_dtype not in (*_KIND, None):
            raise ValueError("x_dtype and residual_dtype must be bfloat16 or float32")
        self.n, self.d, self.payload = n, d, payload
        self.device = _device(device)
        check_tensor("weight", weight, (d,), torch.float32, self.device)
        self.weight = weight
        self.x_dtype, self.residual_dtype = x_dtype, residual_dtype
        self.h_dtype = x_dtype if residual_dtype is None else residual_dtype
        group = PAYLOADS[payload]
        new = dict(device=self.device)
        self.params = abi.NormParams(n, d, d, _KIND[x_dtype], _KIND[self.h_dtype], group or 0, eps)
        self.y = torch.empty((n, d), dtype=torch.bfloat16, **new) \
            if payload == "bf16" or keep_bf16 else None
        self.xq = self.xs = None
        if payload != "bf16":
            self.xq = torch.empty((n, d), dtype=torch.uint8, **new)
            self.xs = torch.empty((n, abi.fp8_scale_groups(d, group)), dtype=torch.float32, **new)
        self.residual_out = None if residual_dtype is None else \
            torch.empty((n, d), dtype=residual_dtype, **new)
        self.rstd = torch.empty((n,), dtype=torch.float32, **new)
        self.dev_status = torch.zeros((1,), dtype=torch.int32, **new)
        self._h = None
        self._grads = None

    @property
    def output(self):
        """What ``MoELayer.forward`` takes: the bf16 rows, or (codes, scales)."""
        return self.y if self.payload == "bf16" else (self.xq, self.xs)

    def forward(self, x, residual=None, stream=None):
        """Returns ``output``; the sum that becomes the residual stream is
        ``residual_out``."""
        abi.check_current_device(self.device)
        check_tensor("x", x, (self.n, self.d), self.x_dtype, self.device, rows_strided=True)
        if (residual is None) != (self.residual_dtype is None):
            raise ValueError("residual must be given exactly when residual_dtype is")
        if residual is not None:
            check_tensor("residual", residual, (self.n, self.d), self.residual_dtype, self.device)
        self.params.x_stride = x.stride(0) if self.n > 1 else self.d
        abi.moe_add_rms_norm(self.params, x, residual, self.weight, self.residual_out, self.y,
                             self.xq, self.xs, self.rstd, self.dev_status, stream)
        # without a residual the backward reads x itself as h
        self._h = self.residual_out if residual is not None else x
        return self.output

    def backward(self, dy, dresidual_out=None, stream=None):
        """Gradients of the last forward: (dx, dresidual or None, dweight).  dy is [n, d]
        bf16 or fp32; dresidual_out the gradient that reaches residual_out from its other
        readers (None: none).  The buffers are the object's own."""
        abi.check_current_device(self.device)
        if self._h is None:
            raise ValueError("backward needs a forward before it")
        if not isinstance(dy, torch.Tensor) or dy.dtype not in _KIND:
            raise ValueError("dy must be bfloat16 or float32")
        check_tensor("dy", dy, (self.n, self.d), dy.dtype, self.device)
        if dresidual_out is not None:
            check_tensor("dresidual_out", dresidual_out, (self.n, self.d), self.h_dtype, self.device)
        if not self._h.is_contiguous():
            raise ValueError("backward needs a contiguous x when there is no residual")
        if self._grads is None:
            new = dict(device=self.device)
            ws_bytes = abi.moe_add_rms_norm_backward_workspace_size(self.params)
            with _memory_of(stream, self.device):
                self._grads = (
                    torch.empty((self.n, self.d), dtype=self.x_dtype, **new),
                    None if self.residual_dtype is None else
                    torch.empty((self.n, self.d), dtype=self.residual_dtype, **new),
                    torch.empty((self.d,), dtype=torch.float32, **new),
                    torch.empty((max(ws_bytes, 16),), dtype=torch.uint8, **new), ws_bytes)
        dx, dres, dw, ws, ws_bytes = self._grads
        abi.moe_add_rms_norm_backward(self.params, _KIND[dy.dtype], dy, self._h, self.weight,
                                      self.rstd, dresidual_out, dx, dres, dw, ws, ws_bytes, stream)
        return dx, dres, dw


class RouterLoss:
    """Balance loss of the batches that a router of these parameters routes.

    ``forward`` fills ``counts`` [n_seq, E], ``seq_tokens`` [n_seq + 1] (live tokens of each
    sequence, then the number of sequences that hold any), ``mean_probs`` [n_seq, E] and
    returns ``loss`` [1]; ``backward`` returns ``dlogits`` [T, E]."""

    def __init__(self, T: int, E: int, k: int, alpha: float,
                 score_fn: int = abi.MOE_SCORE_SOFTMAX, route_scale: float = 1.0, n_seq: int = 1,
                 device="cuda"):
        self.T, self.E, self.k, self.n_seq, self.alpha = T, E, k, n_seq, alpha
        self.device = _device(device)
        self.params = abi.RouteParams(T, E, k, score_fn, 1, 1, route_scale)
        self.ws_bytes = abi.moe_balance_loss_workspace_size(self.params, n_seq)
        if self.ws_bytes == 0:
            raise ValueError("unsupported router shape (E <= 512, k <= min(E, 16), "
                             "1 <= n_seq <= 65535, route_scale > 0 for sigmoid gates)")
        new = dict(device=self.device)
        self.ws = torch.empty((self.ws_bytes,), dtype=torch.uint8, **new)
        self.counts = torch.empty((n_seq, E), dtype=torch.int32, **new)
        self.seq_tokens = torch.empty((n_seq + 1,), dtype=torch.int32, **new)
        self.mean_probs = torch.empty((n_seq, E), dtype=torch.float32, **new)
        self.loss = torch.empty((1,), dtype=torch.float32, **new)
        self.dlogits = torch.empty((T, E), dtype=torch.float32, **new)
        self.dev_status = torch.zeros((1,), dtype=torch.int32, **new)

    def _inputs(self, logits, topk_ids, seq_offsets):
        abi.check_current_device(self.device)
        check_tensor("logits", logits, (self.T, self.E), torch.float32, self.device)
        check_tensor("topk_ids", topk_ids, (self.T, self.k), torch.int32, self.device)
        if seq_offsets is not None:
            check_tensor("seq_offsets", seq_offsets, (self.n_seq + 1,), torch.int32, self.device)
        elif self.n_seq != 1:
            raise ValueError("several sequences need seq_offsets")

    def forward(self, logits, topk_ids, seq_offsets=None, stream=None) -> torch.Tensor:
        self._inputs(logits, topk_ids, seq_offsets)
        abi.moe_balance_loss(self.params, self.n_seq, seq_offsets, logits, topk_ids, self.alpha,
                             self.counts, self.seq_tokens, self.mean_probs, self.loss, self.ws,
                             self.ws_bytes, self.dev_status, stream)
        return self.loss

    def backward(self, logits, topk_ids, seq_offsets=None, gates=None, dgates=None, dloss=None,
                 stream=None) -> torch.Tensor:
        """After ``forward`` on the same batch.  dloss: the loss's upstream gradient (fp32 [1],
        None = 1).  With dgates [T, k] (``moe_combine_backward``) and the router's gates the
        gates' gradient is added."""
        self._inputs(logits, topk_ids, seq_offsets)
        if (gates is None) != (dgates is None):
            raise ValueError("gates and dgates go together")
        if dgates is not None:
            check_tensor("gates", gates, (self.T, self.k), torch.float32, self.device)
            check_tensor("dgates", dgates, (self.T, self.k), torch.float32, self.device)
        if dloss is not None:
            check_tensor("dloss", dloss, (1,), torch.float32, self.device)
        abi.moe_route_backward(self.params, self.n_seq, seq_offsets, logits, topk_ids, gates,
                               dgates, self.alpha, self.counts, self.seq_tokens, dloss,
                               self.dlogits, self.dev_status, stream)
        return self.dlogits
