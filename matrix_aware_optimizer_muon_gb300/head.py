"""The operators at a model's head: layer norm and RMS norm, linear cross entropy and log
probabilities, AdamW with 8-bit moments.

Muon takes the blocks' matrices; the norms and the vocabulary matrix stay on AdamW.  The
functions here (same names as the C ABI in include/muon.h) compute the part of a training
step those parameters belong to: the norm before the vocabulary matrix, the loss over the
vocabulary (or its tokens' log probabilities, entropies and alternatives) without keeping
its logits, their gradients, and the update.  Like the rest of the package they only
marshal arguments: every computation runs in the library's kernels.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Dict, List, Optional, Sequence, Tuple, Union

import numpy as np
import torch

from . import _lib
from ._lib import _check, _dt, load_library

ADAMW8_BLOCK = 128

# The current stream's handle without building a Stream object (3 us of a small call's 12).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_here = contextlib.nullcontext()
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_current(*tensors: Optional[torch.Tensor]) -> None:
    """The library launches on the current device: a tensor of another one is refused, for its
    address (and its device's stream) means something else there."""
    here = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError("tensors must be on the current CUDA device")


def _on(stream):
    """Outputs are allocated on the stream they are written on."""
    if stream is None:
        return _here
    if not isinstance(stream, torch.cuda.Stream):   # a handle; ExternalStream(0) would be a new stream
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _stream(stream, t: torch.Tensor) -> int:
    if stream is None and _raw_stream is not None:
        return _raw_stream(t.get_device())
    return _lib._stream(stream)


def _rows(t: torch.Tensor, name: str) -> Tuple[int, int]:
    """(pointer, elements between rows) of a 2-D tensor with contiguous columns."""
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    n, d = t.shape
    ld, one = t.stride()
    if d > 1 and one != 1:
        raise ValueError(f"{name} must have contiguous columns")
    if n > 1 and ld < d:
        raise ValueError(f"{name} must have rows that do not overlap")
    return t.data_ptr(), (ld if n > 1 else max(ld, d))


def _vector(t: Optional[torch.Tensor], n: int, dtype, name: str) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous vector of {n} elements")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    return t.data_ptr()


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def muon_layernorm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                           bias: Optional[torch.Tensor] = None, eps: float = 1e-5, stream=None):
    """y = (x - mean)*rstd*weight + bias over the last dimension of the 2-D x (rows may be
    strided).  Returns (y, mean, rstd): y contiguous in x's dtype, mean and rstd fp32."""
    px, ldx = _rows(x, "x")
    n, d = x.shape
    pw, pb = _vector(weight, d, None, "weight"), _vector(bias, d, weight.dtype if weight is not None else None, "bias")
    _on_current(x, weight, bias)
    wdt = _dt(weight if weight is not None else bias if bias is not None else x)
    with _on(stream):
        y = torch.empty((n, d), dtype=x.dtype, device=x.device)
        mean = torch.empty(n, dtype=torch.float32, device=x.device)
        rstd = torch.empty(n, dtype=torch.float32, device=x.device)
    _check("muon_layernorm_forward", load_library().muon_layernorm_forward(
        px, ldx, pw, pb, n, d, _dt(x), wdt, eps, y.data_ptr(), d, mean.data_ptr(), rstd.data_ptr(), _stream(stream, x)))
    return y, mean, rstd


def alloc_layernorm_workspace(rows: int, dim: int, device=None) -> torch.Tensor:
    """Workspace of muon_layernorm_backward for these sizes; one call at a time uses it."""
    v = load_library().muon_layernorm_workspace_size(int(rows), int(dim))
    if v == ctypes.c_size_t(-1).value:
        raise _lib.MuonError("muon_layernorm_workspace_size", _lib.MUON_ERR_INVALID)
    return torch.empty(int(v), dtype=torch.uint8, device=device or "cuda")


def muon_layernorm_backward(dy: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor], mean: torch.Tensor,
                            rstd: torch.Tensor, ws: Optional[torch.Tensor] = None,
                            bias: Union[bool, torch.dtype] = True, stream=None, weight_grad: bool = True):
    """Gradients of muon_layernorm_forward: (dx, dweight, dbias).  dweight is None without a
    weight or weight_grad, dbias when bias is False; with neither no workspace is needed.  Without a weight, bias may be the bias's dtype
    (x's if it is True); with one it has the weight's."""
    px, ldx = _rows(x, "x")
    py, ldy = _rows(dy, "dy")
    n, d = x.shape
    if tuple(dy.shape) != (n, d) or dy.dtype != x.dtype:
        raise ValueError("dy and x must have the same shape and dtype")
    pw = _vector(weight, d, None, "weight")
    pm, pr = _vector(mean, n, torch.float32, "mean"), _vector(rstd, n, torch.float32, "rstd")
    _on_current(dy, x, weight, mean, rstd, ws)
    wt = weight.dtype if weight is not None else bias if isinstance(bias, torch.dtype) else x.dtype
    if isinstance(bias, torch.dtype) and bias != wt:
        raise TypeError(f"bias must be {wt}")
    with _on(stream):
        dx = torch.empty((n, d), dtype=x.dtype, device=x.device)
        dw = torch.empty(d, dtype=wt, device=x.device) if weight is not None and weight_grad else None
        db = torch.empty(d, dtype=wt, device=x.device) if bias else None
    _check("muon_layernorm_backward", load_library().muon_layernorm_backward(
        py, ldy, px, ldx, pw, pm, pr, n, d, _dt(x), _dt(weight if weight is not None else db if db is not None else x),
        dx.data_ptr(), d,
        None if dw is None else dw.data_ptr(), None if db is None else db.data_ptr(), _lib._ptr(ws),
        0 if ws is None else ws.numel(), _stream(stream, x)))
    return dx, dw, db


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------
RMS_GROUP = 128


def _like(t: torch.Tensor) -> torch.Tensor:
    """A contiguous tensor of t's shape, dtype and device (a third of torch.empty's time)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _rms_forward(x, weight, residual, eps, need_total, eight, need_y, stream):
    px, ldx = _rows(x, "x")
    n, d = x.shape
    pr, ldr = None, 0
    if residual is not None:
        pr, ldr = _rows(residual, "residual")
        if residual.shape != x.shape or residual.dtype != x.dtype:
            raise ValueError("x and residual must have the same shape and dtype")
    pw = _vector(weight, d, None, "weight")
    _on_current(x, weight, residual)
    codes = scales = y = None
    with _on(stream):
        rstd = torch.empty(n, dtype=torch.float32, device=x.device)
        total = _like(x) if residual is not None and need_total else None
        if need_y:
            y = _like(x)
        if eight:
            codes = torch.empty((n, d), dtype=torch.float8_e4m3fn, device=x.device)
            scales = torch.empty((n, -(-d // RMS_GROUP)), dtype=torch.float32, device=x.device)
    _check("muon_rmsnorm_forward", load_library().muon_rmsnorm_forward(
        px, ldx, pr, ldr, pw, n, d, _dt(x), _dt(x if weight is None else weight), eps,
        None if total is None else total.data_ptr(), d, None if y is None else y.data_ptr(), d,
        None if codes is None else codes.data_ptr(), d, None if scales is None else scales.data_ptr(), rstd.data_ptr(),
        _stream(stream, x)))
    return y, codes, scales, rstd, total if residual is not None else x


def muon_rmsnorm_forward(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                         residual: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None,
                         need_total: bool = True):
    """y = total*rstd*weight over the last dimension of total = x + residual (2-D, rows may be
    strided).  Returns (y, rstd, total): y and total contiguous in x's dtype, rstd fp32.  total is
    x without a residual, and None with one when need_total is False."""
    y, _, _, rstd, total = _rms_forward(x, weight, residual, eps, need_total, False, True, stream)
    return y, rstd, total


def muon_rmsnorm_forward_fp8(x: torch.Tensor, weight: Optional[torch.Tensor] = None,
                             residual: Optional[torch.Tensor] = None, eps: float = 1e-6, stream=None,
                             need_total: bool = True):
    """The same with y in 8 bits.  Returns (codes, scales, rstd, total): codes float8_e4m3fn (rows x
    dim), scales fp32 (rows x ceil(dim/128)); codes[r, c]*scales[r, c//128] stands for y[r, c]."""
    _, codes, scales, rstd, total = _rms_forward(x, weight, residual, eps, need_total, True, False, stream)
    return codes, scales, rstd, total


def alloc_rmsnorm_workspace(rows: int, dim: int, device=None) -> torch.Tensor:
    """Workspace of muon_rmsnorm_backward for these sizes; one call at a time uses it."""
    v = load_library().muon_rmsnorm_workspace_size(int(rows), int(dim))
    if v == ctypes.c_size_t(-1).value:
        raise _lib.MuonError("muon_rmsnorm_workspace_size", _lib.MUON_ERR_INVALID)
    return torch.empty(int(v), dtype=torch.uint8, device=device or "cuda")


def muon_rmsnorm_backward(dy: torch.Tensor, total: torch.Tensor, weight: Optional[torch.Tensor], rstd: torch.Tensor,
                          ws: Optional[torch.Tensor] = None, dtotal: Optional[torch.Tensor] = None, stream=None,
                          weight_grad: bool = True):
    """Gradients of muon_rmsnorm_forward: (dx, dweight).  dx is the gradient of x and of the
    residual alike; dtotal, if given, is the one that total has from elsewhere.  dweight is None
    without a weight or weight_grad; then no workspace is needed."""
    pt, ldt = _rows(total, "total")
    py, ldy = _rows(dy, "dy")
    n, d = total.shape
    if tuple(dy.shape) != (n, d) or dy.dtype != total.dtype:
        raise ValueError("dy and total must have the same shape and dtype")
    pd, ldd = None, 0
    if dtotal is not None:
        pd, ldd = _rows(dtotal, "dtotal")
        if tuple(dtotal.shape) != (n, d) or dtotal.dtype != total.dtype:
            raise ValueError("dtotal and total must have the same shape and dtype")
    pw, pr = _vector(weight, d, None, "weight"), _vector(rstd, n, torch.float32, "rstd")
    _on_current(dy, total, weight, rstd, ws, dtotal)
    with _on(stream):
        dx = _like(total)
        dw = _like(weight) if weight is not None and weight_grad else None
    _check("muon_rmsnorm_backward", load_library().muon_rmsnorm_backward(
        py, ldy, pt, ldt, pw, pr, pd, ldd, n, d, _dt(total), _dt(total if weight is None else weight), dx.data_ptr(), d,
        None if dw is None else dw.data_ptr(), _lib._ptr(ws), 0 if ws is None else ws.numel(), _stream(stream, total)))
    return dx, dw


# ---------------------------------------------------------------------------
# linear cross entropy
# ---------------------------------------------------------------------------
class MuonLinearCe(ctypes.Structure):
    _fields_ = [("H", ctypes.c_void_p), ("W", ctypes.c_void_p), ("labels", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("ldh", ctypes.c_int64), ("ldw", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("ignore_index", ctypes.c_int64)]


def _workspace(nbytes: int, device) -> torch.Tensor:
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")
    _lib.muon_workspace_init(ws)
    return ws


def _ce_args(h: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, ignore_index: int) -> MuonLinearCe:
    ph, ldh = _rows(h, "h")
    pw, ldw = _rows(w, "w")
    if h.dtype != w.dtype or h.shape[1] != w.shape[1]:
        raise ValueError("h and w must have the same dtype and width")
    pl = _vector(labels, h.shape[0], torch.int64, "labels")
    return MuonLinearCe(ph, pw, pl, h.shape[0], w.shape[0], h.shape[1], ldh, ldw, _dt(h), ignore_index)


def muon_linear_ce_workspace_size(rows: int, vocab: int, dim: int, dtype=torch.bfloat16, backward: bool = True,
                                  ldh: Optional[int] = None, ldw: Optional[int] = None) -> int:
    a = MuonLinearCe(None, None, None, rows, vocab, dim, ldh or dim, ldw or dim,
                     _lib.MUON_DTYPE_F32 if dtype == torch.float32 else _lib.MUON_DTYPE_BF16, -100)
    return _ce_workspace_size(a, backward)


def _ce_workspace_size(a: MuonLinearCe, backward: bool) -> int:
    v = load_library().muon_linear_ce_workspace_size(ctypes.byref(a), 1 if backward else 0)
    if v == ctypes.c_size_t(-1).value:
        raise _lib.MuonError("muon_linear_ce_workspace_size", _lib.MUON_ERR_INVALID)
    return int(v)


def linear_ce_workspace_for(h: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, backward: bool = True) -> torch.Tensor:
    """Workspace for these very tensors (their strides and alignment included)."""
    _on_current(h, w, labels)
    return _workspace(_ce_workspace_size(_ce_args(h, w, labels, -100), backward), h.device)


def alloc_linear_ce_workspace(rows: int, vocab: int, dim: int, dtype=torch.bfloat16, backward: bool = True,
                              ldh: Optional[int] = None, ldw: Optional[int] = None, device=None) -> torch.Tensor:
    """Workspace of muon_linear_ce_forward and, with backward, muon_linear_ce_backward.
    ldh and ldw: elements between rows of h and w where they are not contiguous."""
    return _workspace(muon_linear_ce_workspace_size(rows, vocab, dim, dtype, backward, ldh, ldw), device)


def muon_linear_ce_forward(h: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, ws: torch.Tensor,
                           ignore_index: int = -100, stream=None):
    """Cross entropy of the logits h w^T (h: rows x dim, w: vocab x dim) against int64 labels,
    without keeping the logits.  Returns (loss, lse, stats), fp32: each row's loss (0 where
    the label is ignore_index) and log-sum-exp, and [mean loss of the other rows, their count]."""
    a = _ce_args(h, w, labels, ignore_index)
    _on_current(h, w, labels, ws)
    n = h.shape[0]
    with _on(stream):
        loss = torch.empty(n, dtype=torch.float32, device=h.device)
        lse = torch.empty(n, dtype=torch.float32, device=h.device)
        stats = torch.empty(2, dtype=torch.float32, device=h.device)
    _check("muon_linear_ce_forward", load_library().muon_linear_ce_forward(
        ctypes.byref(a), loss.data_ptr(), lse.data_ptr(), stats.data_ptr(), _lib._ptr(ws), ws.numel(), _stream(stream, h)))
    return loss, lse, stats


def muon_linear_ce_backward(h: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor,
                            ws: torch.Tensor, row_grad: Optional[torch.Tensor] = None,
                            stats: Optional[torch.Tensor] = None, upstream: Optional[torch.Tensor] = None,
                            grad_scale: float = 1.0, ignore_index: int = -100, need_dh: bool = True,
                            need_dw: bool = True, stream=None):
    """(dh, dw) of sum_r c_r*loss[r], c_r = grad_scale * upstream * row_grad[r] / stats[1] (each
    factor 1 where it is None; upstream is one fp32 number on the device): with the forward
    pass's stats, the gradient of the mean loss."""
    a = _ce_args(h, w, labels, ignore_index)
    n = h.shape[0]
    pl = _vector(lse, n, torch.float32, "lse")
    pg, ps = _vector(row_grad, n, torch.float32, "row_grad"), _vector(stats, 2, torch.float32, "stats")
    pu = None if upstream is None else _vector(upstream.view(-1), 1, torch.float32, "upstream")
    _on_current(h, w, labels, lse, ws, row_grad, stats, upstream)
    with _on(stream):
        dh = torch.empty((n, h.shape[1]), dtype=h.dtype, device=h.device) if need_dh else None
        dw = torch.empty(tuple(w.shape), dtype=w.dtype, device=h.device) if need_dw else None
    _check("muon_linear_ce_backward", load_library().muon_linear_ce_backward(
        ctypes.byref(a), pl, pg, ps, pu, grad_scale, None if dh is None else dh.data_ptr(),
        None if dw is None else dw.data_ptr(), _lib._ptr(ws), ws.numel(), _stream(stream, h)))
    return dh, dw


# ---------------------------------------------------------------------------
# log probabilities, entropies and alternatives
# ---------------------------------------------------------------------------
LOGPROB_MAX_TOP = 32


def _logprob_args(h: torch.Tensor, w: torch.Tensor, tokens: Optional[torch.Tensor], ignore_index: int) -> MuonLinearCe:
    if tokens is not None:
        return _ce_args(h, w, tokens, ignore_index)
    ph, ldh = _rows(h, "h")
    pw, ldw = _rows(w, "w")
    if h.dtype != w.dtype or h.shape[1] != w.shape[1]:
        raise ValueError("h and w must have the same dtype and width")
    return MuonLinearCe(ph, pw, None, h.shape[0], w.shape[0], h.shape[1], ldh, ldw, _dt(h), ignore_index)


def _logprob_workspace_size(a: MuonLinearCe, top: int, backward: bool) -> int:
    v = load_library().muon_linear_logprob_workspace_size(ctypes.byref(a), int(top), 1 if backward else 0)
    if v == ctypes.c_size_t(-1).value:
        raise _lib.MuonError("muon_linear_logprob_workspace_size", _lib.MUON_ERR_INVALID)
    return int(v)


def alloc_linear_logprob_workspace(rows: int, vocab: int, dim: int, dtype=torch.bfloat16, top: int = 0,
                                   backward: bool = True, ldh: Optional[int] = None, ldw: Optional[int] = None,
                                   device=None) -> torch.Tensor:
    """Workspace of muon_linear_logprob_forward with up to `top` alternatives and, with backward,
    muon_linear_logprob_backward.  ldh and ldw: elements between rows of h and w where they are
    not contiguous."""
    a = MuonLinearCe(None, None, None, rows, vocab, dim, ldh or dim, ldw or dim,
                     _lib.MUON_DTYPE_F32 if dtype == torch.float32 else _lib.MUON_DTYPE_BF16, -100)
    return _workspace(_logprob_workspace_size(a, top, backward), device)


def linear_logprob_workspace_for(h: torch.Tensor, w: torch.Tensor, tokens: Optional[torch.Tensor], top: int = 0,
                                 backward: bool = True) -> torch.Tensor:
    """Workspace for these very tensors (their strides and alignment included)."""
    a = _logprob_args(h, w, tokens, -100)
    _on_current(h, w, tokens)
    return _workspace(_logprob_workspace_size(a, top, backward), h.device)


def muon_linear_logprob_forward(h: torch.Tensor, w: torch.Tensor, tokens: Optional[torch.Tensor], ws: torch.Tensor,
                                top: int = 0, ignore_index: int = -100, stream=None):
    """Log probabilities of int64 tokens under the softmax of the logits h w^T (h: rows x dim, w:
    vocab x dim), the rows' entropies and their `top` (at most 32) likeliest entries, without
    keeping the logits.  Returns (logprob, entropy, lse, ids, alternatives): fp32 but for the int64
    ids; ids and alternatives (their log probabilities) are rows x top, or None with top == 0.
    Rows with token ignore_index give 0, 0, their log-sum-exp, -1 and -inf.  tokens may be None:
    every row counts, and logprob is None."""
    a = _logprob_args(h, w, tokens, ignore_index)
    _on_current(h, w, tokens, ws)
    n, dev, ids, alternatives, logprob = h.shape[0], h.device, None, None, None
    with _on(stream):
        if tokens is not None:
            logprob = torch.empty(n, dtype=torch.float32, device=dev)
        entropy = torch.empty(n, dtype=torch.float32, device=dev)
        lse = torch.empty(n, dtype=torch.float32, device=dev)
        if top > 0:
            ids = torch.empty((n, top), dtype=torch.int64, device=dev)
            alternatives = torch.empty((n, top), dtype=torch.float32, device=dev)
    _check("muon_linear_logprob_forward", load_library().muon_linear_logprob_forward(
        ctypes.byref(a), int(top), None if logprob is None else logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(),
        None if ids is None else ids.data_ptr(), None if alternatives is None else alternatives.data_ptr(),
        _lib._ptr(ws), ws.numel(), _stream(stream, h)))
    return logprob, entropy, lse, ids, alternatives


def muon_linear_logprob_backward(h: torch.Tensor, w: torch.Tensor, tokens: torch.Tensor, lse: torch.Tensor,
                                 entropy: Optional[torch.Tensor], ws: torch.Tensor,
                                 g_logprob: Optional[torch.Tensor] = None, g_entropy: Optional[torch.Tensor] = None,
                                 ignore_index: int = -100, need_dh: bool = True, need_dw: bool = True, stream=None):
    """(dh, dw) of sum_r g_logprob[r]*logprob[r] + g_entropy[r]*entropy[r], with the forward pass's
    lse and entropy; a gradient that is None counts as zeros."""
    a = _ce_args(h, w, tokens, ignore_index)
    n = h.shape[0]
    pl, pe = _vector(lse, n, torch.float32, "lse"), _vector(entropy, n, torch.float32, "entropy")
    pg, ph = _vector(g_logprob, n, torch.float32, "g_logprob"), _vector(g_entropy, n, torch.float32, "g_entropy")
    _on_current(h, w, tokens, lse, entropy, ws, g_logprob, g_entropy)
    with _on(stream):
        dh = torch.empty((n, h.shape[1]), dtype=h.dtype, device=h.device) if need_dh else None
        dw = torch.empty(tuple(w.shape), dtype=w.dtype, device=h.device) if need_dw else None
    _check("muon_linear_logprob_backward", load_library().muon_linear_logprob_backward(
        ctypes.byref(a), pl, pe, pg, ph, None if dh is None else dh.data_ptr(), None if dw is None else dw.data_ptr(),
        _lib._ptr(ws), ws.numel(), _stream(stream, h)))
    return dh, dw


# ---------------------------------------------------------------------------
# AdamW with 8-bit moments
# ---------------------------------------------------------------------------
_PARAM8 = np.dtype([("P", "u8"), ("G", "u8"), ("m", "u8"), ("v", "u8"), ("m_scale", "u8"), ("v_scale", "u8"),
                    ("numel", "i8"), ("first", "i8"), ("p_dtype", "i4"), ("g_dtype", "i4")])


class AdamW8:
    """AdamW over a list of parameters, both moments in 8 bits (see muon_adamw8_step in
    include/muon.h for the format).  The state is four flat byte buffers, 2 + 2/128 bytes a
    parameter; parameter i's codes start at self.starts[i], a multiple of 128.  Parameters may be
    of two dtypes (a bf16 matrix beside fp32 norms): those of one dtype stay of one dtype, and
    so do their gradients; each dtype is one launch."""

    def __init__(self, params: Sequence[torch.Tensor], lr: float = 1e-4, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.0, seed: int = 0):
        self.params: List[torch.Tensor] = list(params)
        if not self.params:
            raise ValueError("no parameters")
        self.lr, self.betas, self.eps, self.weight_decay, self.seed = lr, betas, eps, weight_decay, int(seed) & 0xFFFFFFFF
        self.numels = [p.numel() for p in self.params]
        blocks = [-(-n // ADAMW8_BLOCK) for n in self.numels]
        self.starts = [ADAMW8_BLOCK * b for b in np.concatenate([[0], np.cumsum(blocks)]).tolist()]
        dev, total = self.params[0].device, self.starts[-1]
        self.m, self.v = (torch.zeros(total, dtype=torch.uint8, device=dev) for _ in range(2))
        self.m_scale, self.v_scale = (torch.zeros(total // ADAMW8_BLOCK, dtype=torch.uint8, device=dev) for _ in range(2))
        self._state = (self.m.data_ptr(), self.m_scale.data_ptr(), self.v.data_ptr(), self.v_scale.data_ptr())
        self.step_count = 0
        # the array's entries, parameters of one dtype next to each other
        kinds = [p.dtype for p in self.params]
        self._order = [i for k in dict.fromkeys(kinds) for i in range(len(kinds)) if kinds[i] == k]
        ends = np.cumsum([kinds.count(k) for k in dict.fromkeys(kinds)]).tolist()
        self._groups = list(zip([0, *ends], ends))
        self._arr = np.zeros(len(self.params), dtype=_PARAM8)
        at = np.array(self.starts[:-1], dtype=np.int64)[self._order]
        self._arr["m"], self._arr["v"] = self.m.data_ptr() + at, self.v.data_ptr() + at
        self._arr["m_scale"] = self.m_scale.data_ptr() + at // ADAMW8_BLOCK
        self._arr["v_scale"] = self.v_scale.data_ptr() + at // ADAMW8_BLOCK
        self._arr["numel"], self._arr["first"] = [self.numels[i] for i in self._order], at
        self._addr, self._dtypes = self._arr.ctypes.data, None
        self._check(self.params)

    def _check(self, tensors: Sequence[torch.Tensor]) -> Tuple[Sequence[torch.Tensor], List[int]]:
        """Refuses what the kernel cannot read; returns the tensors in the array's order and each
        group's dtype.  One pass of a C function over the list for each property: 9 us for 48
        tensors."""
        T = torch.Tensor
        if list(map(T.numel, tensors)) != self.numels:
            raise ValueError("parameters keep their sizes, and each has one gradient of the same size")
        if not self.m.is_cuda or set(map(T.get_device, tensors)) != {self.m.get_device()}:
            raise ValueError("parameters and gradients are on one CUDA device, the state's")
        _on_current(self.m)
        if len(self._groups) == 1:
            one = len(set(map(T.dtype.__get__, tensors))) == 1
        else:
            tensors = [tensors[i] for i in self._order]
            one = all(len(set(map(T.dtype.__get__, tensors[a:b]))) == 1 for a, b in self._groups)
        if not one or not all(map(T.is_contiguous, tensors)):
            raise ValueError("parameters of one dtype, and their gradients, are contiguous and of one dtype")
        return tensors, [_dt(tensors[a]) for a, _ in self._groups]

    def _point(self, grads: Sequence[torch.Tensor]) -> None:
        """Checks and enters the tensors of a step."""
        arr = self._arr
        # the parameters too: a model may have been cast or moved since the last step
        params, p_dts = self._check(self.params)
        grads, g_dts = self._check(grads)
        if self._dtypes != (p_dts, g_dts):
            for (a, b), p_dt, g_dt in zip(self._groups, p_dts, g_dts):
                arr["p_dtype"][a:b], arr["g_dtype"][a:b] = p_dt, g_dt
            self._dtypes = p_dts, g_dts
        arr["G"] = list(map(torch.Tensor.data_ptr, grads))
        arr["P"] = list(map(torch.Tensor.data_ptr, params))

    def _launch(self, stream) -> None:
        lib, handle = load_library(), _stream(stream, self.m)
        for a, b in self._groups:
            _check("muon_adamw8_step", lib.muon_adamw8_step(
                self._addr + a * _PARAM8.itemsize, b - a, self.step_count + 1, self.lr, self.betas[0], self.betas[1],
                self.eps, self.weight_decay, self.seed, handle))
        self.step_count += 1

    def step(self, grads: Sequence[torch.Tensor], stream=None) -> None:
        """One asynchronous step."""
        self._point(grads)
        self._launch(stream)

    def moments(self, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
        """The values the codes of both moments stand for, as flat bf16 tensors (exact)."""
        _on_current(self.m)
        n = self.m.numel()
        with _on(stream):
            m = torch.empty(n, dtype=torch.bfloat16, device=self.m.device)
            v = torch.empty(n, dtype=torch.bfloat16, device=self.m.device)
        _check("muon_adamw8_unpack", load_library().muon_adamw8_unpack(
            *self._state, n, m.data_ptr(), v.data_ptr(), _stream(stream, self.m)))
        return m, v

    def state_dict(self) -> Dict:
        return {"step": self.step_count, "seed": self.seed, "m": self.m.clone(), "v": self.v.clone(),
                "m_scale": self.m_scale.clone(), "v_scale": self.v_scale.clone()}

    def _saved(self, sd: Dict):
        """(mine, saved) for each buffer of a state, checked."""
        pairs = list(zip((self.m, self.v, self.m_scale, self.v_scale), [sd[k] for k in ("m", "v", "m_scale", "v_scale")]))
        if any(a.shape != b.shape or b.dtype != torch.uint8 for a, b in pairs):
            raise ValueError("state was saved for other parameters")
        return pairs

    def load_state_dict(self, sd: Dict) -> None:
        for a, b in self._saved(sd):
            a.copy_(b)
        self.step_count, self.seed = int(sd["step"]), int(sd["seed"])
