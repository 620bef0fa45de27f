"""The head's operators as differentiable torch functions: what a model's forward pass
calls, with the gradients from the library's backward kernels."""
from __future__ import annotations

import torch

from . import head


def _plain_rows(t: torch.Tensor) -> torch.Tensor:
    """t as the 2-D row layout the kernels read; copies only what they cannot (a broadcast
    gradient, transposed columns)."""
    t = t.reshape(-1, t.shape[-1])
    n, d = t.shape
    return t if (d == 1 or t.stride(1) == 1) and (n == 1 or t.stride(0) >= d) else t.contiguous()


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        rows = _plain_rows(x)
        y, mean, rstd = head.muon_layernorm_forward(rows, weight, bias, eps)
        ctx.save_for_backward(rows, weight, mean, rstd)
        ctx.shape, ctx.bias_dtype = x.shape, None if bias is None else bias.dtype
        return y.view(x.shape)

    @staticmethod
    def backward(ctx, dy):
        rows, weight, mean, rstd = ctx.saved_tensors
        ws = head.alloc_layernorm_workspace(*rows.shape, device=rows.device)
        dx, dw, db = head.muon_layernorm_backward(_plain_rows(dy), rows, weight, mean, rstd, ws,
                                                  bias=ctx.bias_dtype is not None)
        return dx.view(ctx.shape), dw, None if db is None else db.to(ctx.bias_dtype), None


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, labels, ignore_index):
        rows, labels = _plain_rows(h), labels.reshape(-1).contiguous()
        w = _plain_rows(w)
        ws = head.linear_ce_workspace_for(rows, w, labels, backward=False)
        _, lse, stats = head.muon_linear_ce_forward(rows, w, labels, ws, ignore_index)
        ctx.save_for_backward(rows, w, labels, lse, stats)  # stats[1]: the rows that count
        ctx.shape, ctx.ignore_index = h.shape, ignore_index
        return stats[0].clone()

    @staticmethod
    def backward(ctx, grad):
        rows, w, labels, lse, stats = ctx.saved_tensors
        ws = head.linear_ce_workspace_for(rows, w, labels)
        dh, dw = head.muon_linear_ce_backward(
            rows, w, labels, lse, ws, stats=stats, upstream=grad.float(),
            ignore_index=ctx.ignore_index, need_dh=ctx.needs_input_grad[0], need_dw=ctx.needs_input_grad[1])
        return None if dh is None else dh.view(ctx.shape), dw, None, None


def layer_norm(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5) -> torch.Tensor:
    """Layer norm over the last dimension (weight and bias of that size, fp32 or bf16)."""
    return _LayerNorm.apply(x, weight, bias, eps)


def linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, ignore_index: int = -100) -> torch.Tensor:
    """Mean cross entropy of the logits h w^T, which are never kept (h: ... x dim, w: vocab x
    dim, labels: ... int64); 0 when every label is ignore_index."""
    return _LinearCrossEntropy.apply(h, w, labels, ignore_index)
