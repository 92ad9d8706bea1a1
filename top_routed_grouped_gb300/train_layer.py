"""The end of a training step under torch: ``cross_entropy_loss``, ``LMHead``,
``clip_grad_norm_``.

Like the package's other modules these only marshal: the
``torch.autograd.Function`` calls the library's forward and backward on the
current stream and hands their outputs to autograd.  There is no second
derivative: asking for one raises.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from .train import clip_grads, grad_norm, linear_cross_entropy, linear_cross_entropy_backward


class LinearCrossEntropyFunction(torch.autograd.Function):
    """(loss [T], lse [T]) of ``linear_cross_entropy``; lse has no gradient."""

    @staticmethod
    def forward(ctx, hidden, weight, targets, scale, z_loss, ignore_index):
        loss, lse = linear_cross_entropy(hidden, weight, targets, scale, z_loss, ignore_index)
        ctx.save_for_backward(hidden, weight, targets, lse)
        ctx.args = (scale, z_loss, ignore_index)
        ctx.mark_non_differentiable(lse)
        return loss, lse

    @staticmethod
    @once_differentiable
    def backward(ctx, dloss, _dlse=None):
        hidden, weight, targets, lse = ctx.saved_tensors
        dhidden, dweight = linear_cross_entropy_backward(dloss, lse, hidden, weight, targets, *ctx.args)
        return dhidden, dweight, None, None, None, None


def cross_entropy_loss(hidden, weight, targets, scale: float = 1.0, z_loss: float = 0.0, ignore_index: int = -100):
    """Loss [T] float32 of the next token from ``hidden`` [T, D] and the output
    embedding ``weight`` [V, D] (see ``linear_cross_entropy``), differentiable
    in both (the backward computes both gradients, also where one of them is not
    asked for).  Rows that are left out have loss 0: divide the sum by the number
    of the others for their mean."""
    return LinearCrossEntropyFunction.apply(hidden, weight, targets, scale, z_loss, ignore_index)[0]


class LMHead(torch.nn.Module):
    """The output embedding [V, D] with the loss of the next token:
    ``forward(h [T, D], targets [T])`` is loss [T].  ``weight``: a parameter to
    share (a ``TokenEmbedding``'s) instead of one of its own."""

    def __init__(self, vocabulary: int, hidden: int, scale: float = 1.0, z_loss: float = 0.0, ignore_index: int = -100,
                 dtype: torch.dtype = torch.bfloat16, device=None, weight: torch.nn.Parameter | None = None,
                 init_std: float = 0.02):
        super().__init__()
        if weight is None:
            dev = torch.device("cuda") if device is None else torch.device(device)
            weight = torch.nn.Parameter(torch.empty(vocabulary, hidden, dtype=dtype, device=dev).normal_(0.0, init_std))
        elif weight.shape != (vocabulary, hidden):
            raise ValueError(f"weight: [{vocabulary}, {hidden}] expected, got {list(weight.shape)}")
        self.weight = weight
        self.scale, self.z_loss, self.ignore_index = float(scale), float(z_loss), int(ignore_index)

    def forward(self, h: torch.Tensor, targets: torch.Tensor) -> torch.Tensor:
        return cross_entropy_loss(h, self.weight, targets, self.scale, self.z_loss, self.ignore_index)


def clip_grad_norm_(parameters, max_norm: float, eps: float = 1e-6) -> torch.Tensor:
    """Clip the gradients of ``parameters`` (those that have one) in place to a
    global norm of ``max_norm`` and return the norm that they had.  An infinite
    ``max_norm`` only reads it: the gradients stay as they are, whatever it is."""
    parameters = [parameters] if isinstance(parameters, torch.Tensor) else parameters
    grads = [p.grad for p in parameters if p.grad is not None]
    return grad_norm(grads) if max_norm == math.inf else clip_grads(grads, max_norm, eps)
