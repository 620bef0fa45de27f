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
        raise RuntimeError("layer_norm, rms_norm, linear_cross_entropy and linear_logprobs have no second derivatives")


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


class _RmsNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        if residual is not None and residual.shape != x.shape:      # (as rows they might agree)
            raise ValueError("x and residual must have the same shape and dtype")
        y, rstd, total = head.muon_rmsnorm_forward(_plain_rows(x), weight, None if residual is None else _plain_rows(residual), eps)
        ctx.shape, ctx.behind = x.shape, residual is not None
        if residual is None:
            ctx.save_for_backward(x, weight, rstd, total)
            return y.view(x.shape)
        # (total, an output, stands for x and the residual in the graph, too)
        total = total.view(x.shape)
        ctx.save_for_backward(total, weight, rstd)
        return y.view(x.shape), total

    @staticmethod
    def backward(ctx, dy, dtotal=None):
        x, weight, rstd, *rows = ctx.saved_tensors
        total = rows[0] if rows else x
        dw = None
        if dy is None:
            dx = dtotal
        else:
            with torch.no_grad():
                want_w = ctx.needs_input_grad[1]
                rows = _plain_rows(total)
                ws = head.alloc_rmsnorm_workspace(*rows.shape, device=rows.device) if want_w else None
                dx, dw = head.muon_rmsnorm_backward(_plain_rows(dy), rows, weight, rstd, ws,
                                                    None if dtotal is None else _plain_rows(dtotal), weight_grad=want_w)
                dx = dx.view(ctx.shape)
        dx, dw = _once((dx, dw), (dy, dtotal, x, weight))
        return dx, dw, dx if ctx.behind else None, None


class _LinearLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, w, tokens, ignore_index, top):
        ctx.set_materialize_grads(False)
        if tokens.shape != h.shape[:-1] and tokens.dim() > 1 and h.dim() > 2:   # (as rows they might agree)
            raise ValueError("tokens must have h's leading shape, or one of them one dimension of rows")
        rows, flat = _plain_rows(h), tokens.reshape(-1).contiguous()
        plain = _plain_rows(w)
        ws = head.linear_logprob_workspace_for(rows, plain, flat, top, backward=False)
        logprob, entropy, lse, ids, alternatives = head.muon_linear_logprob_forward(rows, plain, flat, ws, top, ignore_index)
        ctx.save_for_backward(h, w, rows, plain, flat, lse, entropy)
        ctx.shape, ctx.ignore_index = h.shape, ignore_index
        out = logprob.view(tokens.shape), entropy.view(tokens.shape)
        if top == 0:
            return out
        ids, alternatives = ids.view(*tokens.shape, top), alternatives.view(*tokens.shape, top)
        ctx.mark_non_differentiable(ids, alternatives)
        return *out, ids, alternatives

    @staticmethod
    def backward(ctx, g_logprob, g_entropy, *_):
        h, w, rows, plain, tokens, lse, entropy = ctx.saved_tensors
        with torch.no_grad():
            flat = [None if g is None else g.float().reshape(-1).contiguous() for g in (g_logprob, g_entropy)]
            ws = head.linear_logprob_workspace_for(rows, plain, tokens)
            dh, dw = head.muon_linear_logprob_backward(
                rows, plain, tokens, lse, entropy, ws, *flat, ignore_index=ctx.ignore_index,
                need_dh=ctx.needs_input_grad[0], need_dw=ctx.needs_input_grad[1])
            dh = None if dh is None else dh.view(ctx.shape)
            dw = None if dw is None else dw.view(w.shape)
        return *_once((dh, dw), (g_logprob, g_entropy, h, w)), None, None, None


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


def rms_norm(x: torch.Tensor, weight=None, residual=None, eps: float = 1e-6):
    """RMS norm over the last dimension (weight of that size, fp32 or bf16).  With a residual of x's
    shape and dtype, returns (the norm of x + residual, x + residual), both differentiable."""
    return _RmsNorm.apply(x, weight, residual, eps)


def linear_logprobs(h: torch.Tensor, w: torch.Tensor, tokens: torch.Tensor, ignore_index: int = -100, top: int = 0):
    """(logprob, entropy) of the softmax of the logits h w^T, which are never kept (h: ... x dim, w:
    vocab x dim, tokens: ... int64, where either may have its rows in one dimension), of the tokens' shape;
    both 0 where a token is ignore_index.
    With top > 0 also (ids, alternatives) of the likeliest entries, ... x top, without gradient."""
    return _LinearLogprobs.apply(h, w, tokens, ignore_index, top)
