"""The global norm of a list of gradients, and clipping by it (muon_clip_grad_norm in
include/muon.h): what a training step does between its backward pass and the optimizer."""
from __future__ import annotations

import math
from typing import Optional, Sequence

import numpy as np
import torch

from . import _lib
from ._lib import _check, load_library
from .head import _on, _on_current, _stream

_GRAD = np.dtype([("G", "u8"), ("numel", "i8"), ("dtype", "i4"), ("reserved", "i4")])


def _code(dtype: torch.dtype) -> int:
    if dtype == torch.bfloat16:
        return _lib.MUON_DTYPE_BF16
    if dtype == torch.float32:
        return _lib.MUON_DTYPE_F32
    raise TypeError(f"unsupported dtype {dtype}")


def alloc_clip_workspace(device=None) -> torch.Tensor:
    """Workspace of muon_clip_grad_norm, for any list; one call at a time uses it."""
    return torch.empty(int(load_library().muon_clip_workspace_size()), dtype=torch.uint8, device=device or "cuda")


def muon_clip_grad_norm(grads: Sequence[torch.Tensor], max_norm: Optional[float], ws: torch.Tensor,
                        stream=None) -> torch.Tensor:
    """Norm over all elements of all gradients (fp32 or bf16, contiguous, of any shapes) as they are;
    where it is above max_norm, they are scaled in place by max_norm/norm.  None or infinity
    computes the norm alone.  Returns the norm, one fp32 number on the device: nothing waits
    for it."""
    T, grads = torch.Tensor, list(grads)
    # one pass of a C function over the list for each property
    if not ws.is_cuda or not set(map(T.get_device, grads)) <= {ws.get_device()}:
        raise ValueError("gradients and workspace must be on one CUDA device")
    _on_current(ws)
    if not all(map(T.is_contiguous, grads)):
        raise ValueError("gradients must be contiguous")
    arr = np.zeros(max(len(grads), 1), dtype=_GRAD)
    if grads:
        kinds = list(map(T.dtype.__get__, grads))
        codes = {k: _code(k) for k in set(kinds)}
        arr["G"], arr["numel"] = list(map(T.data_ptr, grads)), list(map(T.numel, grads))
        arr["dtype"] = [codes[k] for k in kinds] if len(codes) > 1 else codes[kinds[0]]
    with _on(stream):
        norm = torch.empty((), dtype=torch.float32, device=ws.device)
    _check("muon_clip_grad_norm", load_library().muon_clip_grad_norm(
        arr.ctypes.data, len(grads), math.inf if max_norm is None else max_norm, norm.data_ptr(), _lib._ptr(ws),
        ws.numel(), _stream(stream, ws)))
    return norm
