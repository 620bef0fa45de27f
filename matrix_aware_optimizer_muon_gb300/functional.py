"""The head's operators as differentiable torch functions: what a model's forward pass
calls, with the gradients from the library's backward kernels.  The gradients have no
derivative of their own: differentiating them (create_graph) raises RuntimeError."""
from __future__ import annotations

import torch

from . import head


def _plain_rows(t: torch.Tensor) -> torch.Tensor:
    """t as the 2-D row layout the kernels read; copies only what they cannot (a broadcast
    gradient, transposed columns)."""
    t = t.reshape(-1, t.shape[-1])
    n, d = t.shape
    return t if (d == 1 or t.stride(1) == 1) and (n == 1 or t.stride(0) >= d) else t.contiguous()


class _Once(torch.autograd.Function):
    """Passes the first `count` tensors, gradients, on, as functions of them all."""

    @staticmethod
    def forward(ctx, count, *tensors):
        return tuple(None if t is None else t.view_as(t) for t in tensors[:count])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("layer_norm and linear_cross_entropy have no second derivatives")


def _once(grads, depends):
    """The gradients of a backward pass, which came from `depends`.  Without a graph of their own
    they would count as constants, and a penalty on them would be lost without a word."""
    return _Once.apply(len(grads), *grads, *depends) if torch.is_grad_enabled() else grads


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        rows = _plain_rows(x)
        y, mean, rstd = head.muon_layernorm_forward(rows, weight, bias, eps)
        ctx.save_for_backward(x, rows, weight, mean, rstd)
        ctx.shape, ctx.bias_dtype = x.shape, None if bias is None else bias.dtype
        return y.view(x.shape)

    @staticmethod
    def backward(ctx, dy):
        x, rows, weight, mean, rstd = ctx.saved_tensors
        with torch.no_grad():
            # column sums only for what is trained
            want_w, want_b = ctx.needs_input_grad[1:3]
            ws = head.alloc_layernorm_workspace(*rows.shape, device=rows.device) if want_w or want_b else None
            dx, dw, db = head.muon_layernorm_backward(_plain_rows(dy), rows, weight, mean, rstd, ws,
                                                      bias=want_b and ctx.bias_dtype, weight_grad=want_w)
            dx = dx.view(ctx.shape)
        return *_once((dx, dw, db), (dy, x, weight)), None


class _LinearCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, labels, ignore_index):
        rows, labels = _plain_rows(h), labels.reshape(-1).contiguous()
        plain = _plain_rows(w)
        ws = head.linear_ce_workspace_for(rows, plain, labels, backward=False)
        _, lse, stats = head.muon_linear_ce_forward(rows, plain, labels, ws, ignore_index)
        ctx.save_for_backward(h, w, rows, plain, labels, lse, stats)  # stats[1]: the rows that count
        ctx.shape, ctx.ignore_index = h.shape, ignore_index
        return stats[0].clone()

    @staticmethod
    def backward(ctx, grad):
        h, w, rows, plain, labels, lse, stats = ctx.saved_tensors
        with torch.no_grad():
            ws = head.linear_ce_workspace_for(rows, plain, labels)
            dh, dw = head.muon_linear_ce_backward(
                rows, plain, labels, lse, ws, stats=stats, upstream=grad.float(),
                ignore_index=ctx.ignore_index, need_dh=ctx.needs_input_grad[0], need_dw=ctx.needs_input_grad[1])
            dh = None if dh is None else dh.view(ctx.shape)
        return *_once((dh, dw), (grad, h, w)), None, None


def layer_norm(x: torch.Tensor, weight=None, bias=None, eps: float = 1e-5) -> torch.Tensor:
    """Layer norm over the last dimension (weight and bias of that size, fp32 or bf16)."""
    return _LayerNorm.apply(x, weight, bias, eps)


def linear_cross_entropy(h: torch.Tensor, w: torch.Tensor, labels: torch.Tensor, ignore_index: int = -100) -> torch.Tensor:
    """Mean cross entropy of the logits h w^T, which are never kept (h: ... x dim, w: vocab x
    dim, labels: ... int64); 0 when every label is ignore_index."""
    return _LinearCrossEntropy.apply(h, w, labels, ignore_index)
