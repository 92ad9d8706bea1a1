"""The operators around the layer as torch modules: ``TokenEmbedding``,
``BlockNorm``, ``distillation_loss``.

Like ``MoEFunction`` these only marshal: each ``torch.autograd.Function``
calls the library's forward and backward on the current stream and hands
their outputs to autograd.  Gradients of weights come out of the library in
FP32; autograd casts one to its parameter's dtype.  There is no second
derivative: asking for one raises.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from .step import block_norm, block_norm_backward, distill, distill_backward, embed, embed_backward


class EmbedFunction(torch.autograd.Function):
    """out = scale * table[ids]: table [V, H], ids [T]."""

    @staticmethod
    def forward(ctx, table, ids, scale=1.0, padding_id=None, out_dtype=None):
        ctx.save_for_backward(ids)
        ctx.shape, ctx.scale, ctx.padding_id = table.shape[0], scale, padding_id
        return embed(table, ids, scale=scale, out_dtype=out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        return embed_backward(ctx.saved_tensors[0], dout, ctx.shape, scale=ctx.scale,
                              padding_id=ctx.padding_id), None, None, None, None


class BlockNormFunction(torch.autograd.Function):
    """(r_out, h) of ``block_norm``; without y, h alone."""

    @staticmethod
    def forward(ctx, r, y, w_post, w_pre, gate, scale, eps, weight_offset, dtype):
        r_out, h = block_norm(r, y, w_post, w_pre, gate, scale=scale, eps=eps, weight_offset=weight_offset,
                              dtype=dtype)
        ctx.save_for_backward(r_out if w_pre is not None else None, y, w_post, w_pre, gate)
        ctx.args = dict(scale=scale, eps=eps, weight_offset=weight_offset)
        ctx.set_materialize_grads(False)
        if y is None:
            return h
        return r_out if h is None else (r_out, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        r_out, y, w_post, w_pre, gate = ctx.saved_tensors
        dr_out = grads[0] if y is not None else None
        dh = grads[-1] if w_pre is not None else None
        if dr_out is None and dh is None:
            return (None,) * 9
        if w_pre is not None and dh is None:  # nothing came through h
            dh = torch.zeros_like(r_out, dtype=y.dtype)
        d = block_norm_backward(dr_out, dh, r_out, y, w_post, w_pre, gate, **ctx.args)
        return d["dr"], d["dy"], d["dw_post"], d["dw_pre"], d["dgate"], None, None, None, None


class DistillFunction(torch.autograd.Function):
    """loss [T] of ``distill``; the teacher gets no gradient."""

    @staticmethod
    def forward(ctx, logits, t_ids, t_logits, temperature, scale, t_lse):
        loss, lse = distill(logits, t_ids, t_logits, temperature, scale, t_lse)
        ctx.save_for_backward(logits, t_ids, t_logits, t_lse, lse)
        ctx.args = (temperature, scale)
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss):
        logits, t_ids, t_logits, t_lse, lse = ctx.saved_tensors
        return distill_backward(dloss, lse, logits, t_ids, t_logits, *ctx.args, t_lse), None, None, None, None, None


def distillation_loss(logits, t_ids, t_logits, temperature: float = 1.0, scale: float = 1.0, t_lse=None):
    """Loss [T] float32 of the student's ``logits`` [T, V] against the
    teacher's top logits (see ``distill``), differentiable in ``logits`` (by
    ``distill_backward``, with its limit)."""
    return DistillFunction.apply(logits, t_ids, t_logits, temperature, scale, t_lse)


class TokenEmbedding(torch.nn.Module):
    """A table [V, H] whose rows leave scaled: ``forward(ids [T])`` is [T, H].
    ``padding_id``: a token without gradient, counted from the end where it is
    negative."""

    def __init__(self, num_embeddings: int, hidden: int, scale: float = 1.0, padding_id: int | None = None,
                 dtype: torch.dtype = torch.bfloat16, out_dtype: torch.dtype | None = None, device=None,
                 init_std: float = 0.02):
        super().__init__()
        if padding_id is not None:
            if not -num_embeddings <= padding_id < num_embeddings:
                raise ValueError(f"padding_id {padding_id}: not one of {num_embeddings} tokens")
            padding_id %= num_embeddings
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.weight = torch.nn.Parameter(torch.empty(num_embeddings, hidden, dtype=dtype, device=dev).normal_(0.0, init_std))
        self.scale, self.padding_id, self.out_dtype = float(scale), padding_id, out_dtype

    def forward(self, ids: torch.Tensor) -> torch.Tensor:
        return EmbedFunction.apply(self.weight, ids, self.scale, self.padding_id, self.out_dtype)


class BlockNorm(torch.nn.Module):
    """What stands between two blocks: ``forward(r, y, gate)`` takes the residual
    rows and the block's output and returns (r_out, h); ``forward(r)`` is the
    norm before the first block and returns h.

    ``post`` / ``pre``: whether there is a norm after the block / before the
    next one (without the latter ``forward`` returns r_out alone).  Weights
    are stored as w - weight_offset."""

    def __init__(self, hidden: int, post: bool = True, pre: bool = True, scale: float = 1.0, eps: float = 1e-6,
                 weight_offset: float = 0.0, dtype: torch.dtype = torch.bfloat16, device=None):
        super().__init__()
        dev = torch.device("cuda") if device is None else torch.device(device)
        mk = lambda: torch.nn.Parameter(torch.full((hidden,), 1.0 - weight_offset, dtype=dtype, device=dev))  # noqa: E731
        self.w_post = mk() if post else None
        self.w_pre = mk() if pre else None
        self.scale, self.eps, self.weight_offset = float(scale), float(eps), float(weight_offset)

    def forward(self, r: torch.Tensor, y: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                dtype: torch.dtype | None = None):
        return BlockNormFunction.apply(r, y, self.w_post if y is not None else None, self.w_pre, gate, self.scale,
                                       self.eps, self.weight_offset, dtype)
