"""Binding of the end of a training step: the loss of the next token from
hidden rows, the gradients' norm and clipping.

Like ``step.py`` this module only marshals: torch supplies device memory and
the stream, the library's CUDA kernels do every step (contracts in
``include/moe.h``).  ``moe_*`` functions mirror the C entry points;
``linear_cross_entropy`` with its gradient and step, ``grad_norm``,
``clip_grads`` and ``scale_grads`` take tensors, check them, allocate the
outputs and call.
"""
from __future__ import annotations

import struct

import torch

from . import _check, lib
from .step import _ids, _like, _on, _ptr, _row_type, _rows, _same_or_f32, _vec, _written, _ws

_CE = struct.Struct("7i2fi4q8Q")     # moe_linear_ce_args_t
_GRADS = struct.Struct("2i5Q2fQ")    # moe_grads_args_t
LOSS, GRAD, STEP = 1, 2, 3


# ---------------------------------------------------------------- raw ABI
def moe_linear_ce(args: bytes, ws, ws_bytes: int, stream) -> None:
    _check("moe_linear_ce", lib().moe_linear_ce(args, ws, ws_bytes, stream))


def moe_linear_ce_workspace_size(args: bytes, call: int) -> int:
    return lib().moe_linear_ce_workspace_size(args, call)


def moe_linear_ce_backward(args: bytes, ws, ws_bytes: int, stream) -> None:
    _check("moe_linear_ce_backward", lib().moe_linear_ce_backward(args, ws, ws_bytes, stream))


def moe_linear_ce_step(args: bytes, ws, ws_bytes: int, stream) -> None:
    _check("moe_linear_ce_step", lib().moe_linear_ce_step(args, ws, ws_bytes, stream))


def moe_grad_norm(args: bytes, ws, ws_bytes: int, stream) -> None:
    _check("moe_grad_norm", lib().moe_grad_norm(args, ws, ws_bytes, stream))


def moe_grad_workspace_size(args: bytes) -> int:
    return lib().moe_grad_workspace_size(args)


def moe_grad_clip(args: bytes, ws, ws_bytes: int, stream) -> None:
    _check("moe_grad_clip", lib().moe_grad_clip(args, ws, ws_bytes, stream))


def moe_grad_scale(args: bytes, stream) -> None:
    _check("moe_grad_scale", lib().moe_grad_scale(args, stream))


# ---------------------------------------------------------------- linear cross entropy
def _linear_ce(stream, hidden, weight, targets, scale, z_loss, ignore_index, dloss, lse, dweight, dweight_dtype, ws,
               mode):
    if hidden.dim() != 2 or weight.dim() != 2:
        raise ValueError("hidden: [T, D] and weight: [V, D] expected")
    T, V, D = hidden.shape[0], *weight.shape
    dtype, device, dev = weight.dtype, hidden.device, hidden.get_device()
    code = _row_type(dtype, "weight")
    given = hidden
    hidden, ld_h = _rows(hidden, T, D, dtype, dev, "hidden")
    weight, ld_w = _rows(weight, V, D, dtype, dev, "weight")
    if targets.dim() != 1 or targets.shape[0] != T:
        raise ValueError(f"targets: [{T}] expected, got {list(targets.shape)}")
    targets = _ids(targets, dev)
    loss, dhidden, gcode, accumulate, ld_dh = None, None, code, dweight is not None, 0
    if mode & LOSS:
        loss = torch.empty(T, dtype=torch.float32, device=device)
    if mode == LOSS:
        lse = torch.empty(T, dtype=torch.float32, device=device)
    elif mode == GRAD:
        lse = _vec(lse, T, (torch.float32,), dev, "lse")
    if mode & GRAD:
        dloss = _vec(dloss, T, (torch.float32,), dev, "dloss")
        dhidden = torch.empty_like(given, memory_format=torch.contiguous_format)
        if accumulate:
            if dweight.dtype is not torch.float32 or dweight.shape != (V, D) or not dweight.is_contiguous() or \
                    dweight.get_device() != dev:
                raise ValueError(f"dweight: contiguous float32 [{V}, {D}] on device {dev} expected")
            gcode = 0
        else:
            dweight_dtype = dtype if dweight_dtype is None else dweight_dtype
            gcode = _same_or_f32(dtype, dweight_dtype, "dweight_dtype")
            dweight = torch.empty((V, D), dtype=dweight_dtype, device=device)
    args = _CE.pack(T, D, V, code, gcode, accumulate, targets.dtype is torch.int64, scale, z_loss, 0, ignore_index, ld_h,
                    ld_w, ld_dh, hidden.data_ptr(), weight.data_ptr(), targets.data_ptr(), _ptr(dloss), _ptr(loss),
                    _ptr(lse), _ptr(dhidden), _ptr(dweight))
    ws, n = _ws(moe_linear_ce_workspace_size(args, mode) if ws is None else 0, ws, device)
    (moe_linear_ce, moe_linear_ce_backward, moe_linear_ce_step)[mode - 1](args, ws.data_ptr(), n, stream)
    if accumulate:
        _written(dweight)
    if mode == LOSS:
        return loss, lse
    return (dhidden, dweight) if mode == GRAD else (loss, dhidden, dweight)


def linear_cross_entropy(hidden, weight, targets, scale: float = 1.0, z_loss: float = 0.0, ignore_index: int = -100,
                         ws=None, stream=None):
    """(loss [T], lse [T]) float32 of the next token from hidden rows, without
    keeping logits: with x_t = scale * weight @ hidden_t,

        lse_t = log sum_v exp(x_tv)      loss_t = lse_t - x_t[target_t] + z_loss * lse_t^2

    hidden [T, D], weight [V, D] (the output embedding, of one type), targets
    [T] int32 or int64.  Rows whose target is ``ignore_index`` are left out:
    they are not read, their loss and lse are 0.  So is a target outside the
    vocabulary, with device status 7."""
    return _on(hidden, stream, _linear_ce, hidden, weight, targets, scale, z_loss, ignore_index, None, None, None, None,
               ws, LOSS)


def linear_cross_entropy_backward(dloss, lse, hidden, weight, targets, scale: float = 1.0, z_loss: float = 0.0,
                                  ignore_index: int = -100, dweight=None, dweight_dtype=None, ws=None, stream=None):
    """(dhidden, dweight) of ``linear_cross_entropy`` for upstream gradients
    ``dloss`` [T] float32 and the forward's lse.  dhidden has hidden's type and
    zeros in the rows that are left out; dweight [V, D] has the weight's type
    or ``dweight_dtype`` (float32), or is the float32 tensor ``dweight``, added to.
    Float32 sums of bfloat16 rows: what goes into their products, dx and the rows
    of hidden, is bfloat16 all the same, rounded once each."""
    return _on(hidden, stream, _linear_ce, hidden, weight, targets, scale, z_loss, ignore_index, dloss, lse, dweight,
               dweight_dtype, ws, GRAD)


def linear_cross_entropy_step(hidden, weight, targets, dloss, scale: float = 1.0, z_loss: float = 0.0,
                              ignore_index: int = -100, dweight=None, dweight_dtype=None, ws=None, stream=None):
    """(loss, dhidden, dweight) in one call: ``linear_cross_entropy`` and
    ``linear_cross_entropy_backward`` where the upstream gradient of each row's
    loss is known beforehand."""
    return _on(hidden, stream, _linear_ce, hidden, weight, targets, scale, z_loss, ignore_index, dloss, None, dweight,
               dweight_dtype, ws, STEP)


# ---------------------------------------------------------------- gradients
def _packer():
    """``pack`` of the native module, which reads tensors as the torch has them that it was built for."""
    from .build import bind_target
    try:
        from . import _tensor_list as m
    except ImportError as e:
        m, why = None, e
    else:
        why = None
    if m is None or getattr(m, "built_for", None) != bind_target():
        raise RuntimeError("_tensor_list.so is missing or of another torch: build it with "
                           "`python -m top_routed_grouped_gb300.build`") from why
    return m.pack


def _pack(grads, out, dev):
    global _pack
    _pack = _packer()
    return _pack(grads, out, dev)


def _grads(stream, grads, out, norm, max_norm, eps, ws, mode):
    dev, device = grads[0].get_device(), grads[0].device
    held, src, dst, numel, code, ocode = _pack(grads, out, dev)
    if mode & 1:
        norm = torch.empty((), dtype=torch.float32, device=device)
    elif norm.dtype is not torch.float32 or norm.numel() != 1 or norm.get_device() != dev:
        raise ValueError(f"norm: one float32 on device {dev} expected")
    args = _GRADS.pack(len(grads), 0, src, dst, numel, code, ocode, max_norm, eps, norm.data_ptr())
    if mode & 1:
        ws, n = _ws(moe_grad_workspace_size(args) if ws is None else 0, ws, device)
        (moe_grad_norm if mode == 1 else moe_grad_clip)(args, ws.data_ptr(), n, stream)
    else:
        moe_grad_scale(args, stream)
    del held
    if mode & 2:
        _written(grads if out is None else out)
    return norm


def _listed(ts, name: str) -> list:
    ts = list(ts)
    if ts and not isinstance(ts[0], torch.Tensor):
        raise ValueError(f"{name}: tensors expected, got {type(ts[0]).__name__}")
    return ts


def grad_norm(grads, ws=None, stream=None):
    """The 2-norm over all elements of ``grads`` (tensors of float32 or
    bfloat16 on one device, in any gapless order), a float32 scalar there.  Its
    last bit may depend on where the tensors lie between 16-byte boundaries."""
    grads = _listed(grads, "grads")
    if not grads:
        return torch.zeros((), dtype=torch.float32, device="cuda")
    return _on(grads[0], stream, _grads, grads, None, None, 0.0, 0.0, ws, 1)


def clip_grads(grads, max_norm: float, eps: float = 1e-6, out=None, ws=None, stream=None):
    """Scale ``grads`` by min(1, max_norm / (norm + eps)) and return the norm
    that they had.  In place, or into ``out``: as many tensors of the same
    sizes, of float32 or bfloat16 (accumulated float32 gradients become their
    parameters' type this way)."""
    grads, out = _listed(grads, "grads"), None if out is None else _listed(out, "out")
    if not grads:
        return grad_norm(grads)
    return _on(grads[0], stream, _grads, grads, out, None, max_norm, eps, ws, 3)


def scale_grads(grads, norm, max_norm: float, eps: float = 1e-6, out=None, stream=None) -> None:
    """``clip_grads`` for a norm [1] float32 that is on the device already: one
    put together from the norms of several ranks, say."""
    grads, out = _listed(grads, "grads"), None if out is None else _listed(out, "out")
    if grads:
        _on(grads[0], stream, _grads, grads, out, norm, max_norm, eps, None, 2)
