"""Binding of the operators around the layer: embedding, block norms, distillation.

Like the package's other bindings this module only marshals: torch supplies
device memory and the stream, the library's CUDA kernels do every step
(contracts in ``include/moe.h``).  ``moe_*`` functions mirror the C entry
points (a packed argument struct in, ``MoEError`` on a non-zero status);
``embed``, ``block_norm`` and ``distill`` with their gradients take tensors,
check them, allocate the outputs and call.  They are short calls (a decoding
step makes many of them), so the structs are packed in one go by
``struct.Struct`` instead of field by field.
"""
from __future__ import annotations

import struct

import torch

from . import _check, lib

_NORM = struct.Struct("6i3fi10q14Q")   # moe_norm_args_t
_EMBED = struct.Struct("6ifi3q5Q")     # moe_embed_args_t
_DISTILL = struct.Struct("4i2f2q8Q")   # moe_distill_args_t
GATE = {"none": 0, "token": 1, "channel": 2, "element": 3}
_DTYPE = {torch.float32: 0, torch.bfloat16: 1}
MAX_SLOTS = 256


# ---------------------------------------------------------------- raw ABI
def moe_block_norm(args: bytes, stream) -> None:
    _check("moe_block_norm", lib().moe_block_norm(args, stream))


def moe_block_norm_workspace_size(args: bytes) -> int:
    return lib().moe_block_norm_workspace_size(args)


def moe_block_norm_backward(args: bytes, ws, ws_bytes: int, stream) -> None:
    _check("moe_block_norm_backward", lib().moe_block_norm_backward(args, ws, ws_bytes, stream))


def moe_embed(args: bytes, stream) -> None:
    _check("moe_embed", lib().moe_embed(args, stream))


def moe_embed_workspace_size(args: bytes) -> int:
    return lib().moe_embed_workspace_size(args)


def moe_embed_backward(args: bytes, ws, ws_bytes: int, stream) -> None:
    _check("moe_embed_backward", lib().moe_embed_backward(args, ws, ws_bytes, stream))


def moe_distill(args: bytes, stream) -> None:
    _check("moe_distill", lib().moe_distill(args, stream))


def moe_distill_backward(args: bytes, stream) -> None:
    _check("moe_distill_backward", lib().moe_distill_backward(args, stream))


def moe_distill_step(args: bytes, stream) -> None:
    _check("moe_distill_step", lib().moe_distill_step(args, stream))


# ---------------------------------------------------------------- helpers
def _on(t: torch.Tensor, stream, call, *args):
    """call(raw stream, *args) with ``t``'s device current and, where a stream
    is given, that stream current too, so that what the call allocates belongs
    to the stream that works on it."""
    if not t.is_cuda:
        raise ValueError("the operators run on CUDA tensors")
    dev = t.get_device()
    if stream is None and dev == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(dev), *args)
    with torch.cuda.device(dev):
        if stream is None:
            return call(torch._C._cuda_getCurrentRawStream(dev), *args)
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=dev)
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream, *args)


def _like(t, ld, dtype=None):
    """Dense rows of the shape of ``t``, whose row stride is ``ld``."""
    if ld:
        return torch.empty_like(t, dtype=dtype, memory_format=torch.contiguous_format)
    return torch.empty_like(t, dtype=dtype)


def _rows(t, T: int, N: int, dtype, dev, name: str):
    """``t`` as [T, N] rows of ``dtype`` with neighbouring channels, and its
    row stride (0 where the rows are dense).  One row of a wider matrix keeps
    that stride, so that it runs as among its neighbours and gets the same bits."""
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != 2 or t.shape[0] != T or t.shape[1] != N:
        raise ValueError(f"{name}: {dtype} [{T}, {N}] on device {dev} expected, got {t.dtype} {list(t.shape)} "
                         f"on device {t.get_device()}")
    if t.is_contiguous():
        return t, t.stride(0) if T == 1 and t.stride(0) > N else 0
    if (N > 1 and t.stride(1) != 1) or t.stride(0) < N:
        return t.contiguous(), 0
    return t, t.stride(0)


def _vec(t, N: int, dtypes, dev, name: str):
    if t.dtype not in dtypes or t.get_device() != dev or t.shape != (N,):
        raise ValueError(f"{name}: [{N}] of {dtypes} on device {dev} expected, got {t.dtype} {list(t.shape)} "
                         f"on device {t.get_device()}")
    return t if t.is_contiguous() else t.contiguous()


def _row_type(dtype, what: str) -> int:
    if dtype not in _DTYPE:
        raise ValueError(f"{what}: float32 or bfloat16 expected, got {dtype}")
    return _DTYPE[dtype]


def _same_or_f32(dtype, other, what: str) -> int:
    """The code of ``other``, which goes with rows of ``dtype``."""
    if other is not dtype and other is not torch.float32:
        raise ValueError(f"{what}: {dtype} or float32 expected, got {other}")
    return _DTYPE[other]


def _ws(n: int, ws, dev):
    if ws is None:
        ws = torch.empty(n, dtype=torch.uint8, device=dev)
    elif ws.get_device() != dev.index:
        raise ValueError("ws: on another device than the rows")
    elif not ws.is_contiguous():  # the bytes that it names need not all be there
        raise ValueError("ws: contiguous memory expected")
    return ws, ws.numel() * ws.element_size()


# A tensor of the caller's was written: autograd learns of it as of any write in
# place, and refuses to use the old values where it has saved them.
_written = torch.autograd.graph.increment_version


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


# ---------------------------------------------------------------- block_norm
def _norm_weights(dtype, H, dev, w_post, w_pre, gate, T):
    """The gate's kind, the weights' type code, the tensors, the gate's stride."""
    kind, ld, wtype = 0, 0, None
    if gate is not None:
        if gate.dim() == 1:
            kind, wtype = 2, gate.dtype
            gate = _vec(gate, H, (dtype, torch.float32), dev, "gate")
        elif gate.dim() == 2 and gate.shape[1] == 1 and (H != 1 or gate.dtype is not dtype):
            kind = 1
            gate, ld = _rows(gate, T, 1, torch.float32, dev, "gate of a token")
            if ld:
                gate, ld = gate.contiguous(), 0
        else:
            kind = 3
            gate, ld = _rows(gate, T, H, dtype, dev, "gate of an element")
    for name, w in (("w_post", w_post), ("w_pre", w_pre)):
        if w is not None:
            if wtype is None:
                wtype = w.dtype
            elif w.dtype is not wtype:
                raise ValueError(f"{name}: w_post, w_pre and a channel gate have one type")
    if wtype is None:
        wtype = dtype
    code = _same_or_f32(dtype, wtype, "weights")
    if w_post is not None:
        w_post = _vec(w_post, H, (wtype,), dev, "w_post")
    if w_pre is not None:
        w_pre = _vec(w_pre, H, (wtype,), dev, "w_pre")
    return kind, code, w_post, w_pre, gate, ld


def _block_norm(stream, r, y, w_post, w_pre, gate, scale, eps, offset, dtype, inplace):
    T, H = r.shape
    dev = r.get_device()
    if y is not None:
        dtype = y.dtype
    elif dtype is None:
        dtype = r.dtype
    code = _row_type(dtype, "rows")
    rcode = _same_or_f32(dtype, r.dtype, "residual rows")
    if y is None and (w_post is not None or gate is not None):
        raise ValueError("w_post and gate belong to y, which is not given")
    if y is None and w_pre is None:
        raise ValueError("neither y nor w_pre: nothing to compute")
    kind, wcode, w_post, w_pre, gate, ld_gate = _norm_weights(dtype, H, dev, w_post, w_pre, gate, T)
    given = r
    r, ld_r = _rows(r, T, H, r.dtype, dev, "r")
    r_out, h, ld_y, ld_out = given, None, 0, 0
    if y is not None:
        y, ld_y = _rows(y, T, H, dtype, dev, "y")
        if inplace:
            if r is not given:
                raise ValueError("r: rows that cannot be written in place")
            ld_out = ld_r
        else:
            r_out = _like(r, ld_r)
    if w_pre is not None:
        h = _like(r, ld_r) if dtype is r.dtype else _like(r, ld_r, dtype) if y is None else _like(y, ld_y)
    moe_block_norm(_NORM.pack(T, H, code, rcode, wcode, kind, scale, eps, offset, 0, ld_r, ld_y, ld_gate, ld_out, 0, 0, 0,
                              0, 0, 0, r.data_ptr(), _ptr(y), _ptr(w_post), _ptr(w_pre), _ptr(gate), _ptr(r_out),
                              _ptr(h), 0, 0, 0, 0, 0, 0, 0), stream)
    if inplace and y is not None:
        _written(given)
    return r_out, h


def block_norm(r, y=None, w_post=None, w_pre=None, gate=None, scale: float = 1.0, eps: float = 1e-6,
               weight_offset: float = 0.0, dtype=None, inplace: bool = False, stream=None):
    """The join between two blocks: (r_out, h) with

        r_out = r + scale * gate * n(y; w_post)      h = n(r_out; w_pre)
        n(v; w) = v / sqrt(mean(v^2) + eps) * (w + weight_offset)

    r [T, H]: the residual rows (y's type, or float32 beside bfloat16 rows);
    y [T, H]: the block's output, or None (h = n(r; w_pre) alone; r_out is r);
    w_post, w_pre [H] or None: without it that norm is left out (no w_pre: h is
    None); gate: None, [T, 1] float32 (one number a token), [H] (one a channel)
    or [T, H] (one an element); dtype: h's type where there is no y;
    ``inplace``: r_out is written over r."""
    return _on(r, stream, _block_norm, r, y, w_post, w_pre, gate, scale, eps, weight_offset, dtype, inplace)


def _block_norm_backward(stream, dr_out, dh, r_out, y, w_post, w_pre, gate, scale, eps, offset, ws):
    ref = y if y is not None else dh
    if ref is None:
        raise ValueError("neither y nor dh: nothing to compute")
    T, H = ref.shape
    dtype, device, dev = ref.dtype, ref.device, ref.get_device()
    code = _row_type(dtype, "rows")
    like = dr_out if dr_out is not None else r_out
    if like is None:
        raise ValueError("dr_out is needed where there is no w_pre")
    rcode = _same_or_f32(dtype, like.dtype, "residual rows")
    if y is None and (w_post is not None or gate is not None):
        raise ValueError("w_post and gate belong to y, which is not given")
    if (w_pre is None) != (dh is None) or (w_pre is not None and r_out is None):
        raise ValueError("dh, w_pre and r_out go together")
    if y is None and w_pre is None:
        raise ValueError("neither y nor w_pre: nothing to compute")
    if dr_out is None and w_pre is None:
        raise ValueError("dr_out is needed where there is no w_pre")
    kind, wcode, w_post, w_pre, gate, ld_gate = _norm_weights(dtype, H, dev, w_post, w_pre, gate, T)
    ld_r = ld_dr = ld_dh = ld_y = 0
    dr, dy, dw_post, dw_pre, dgate = dr_out, None, None, None, None
    if dr_out is not None:
        dr_out, ld_dr = _rows(dr_out, T, H, like.dtype, dev, "dr_out")
    if w_pre is not None:
        r_out, ld_r = _rows(r_out, T, H, like.dtype, dev, "r_out")
        dh, ld_dh = _rows(dh, T, H, dtype, dev, "dh")
        dr = _like(r_out, ld_r)
        dw_pre = torch.empty(H, dtype=torch.float32, device=device)
    else:
        r_out = None
    if y is not None:
        y, ld_y = _rows(y, T, H, dtype, dev, "y")
        dy = _like(y, ld_y)
        if w_post is not None:
            dw_post = torch.empty(H, dtype=torch.float32, device=device)
        if kind == 3:
            dgate = _like(y, ld_y)
        elif kind:
            dgate = torch.empty((T, 1) if kind == 1 else (H,), dtype=torch.float32, device=device)
    args = _NORM.pack(T, H, code, rcode, wcode, kind, scale, eps, offset, 0, 0, ld_y, ld_gate, ld_r, 0, ld_dr, ld_dh,
                      0, 0, 0, 0, _ptr(y), _ptr(w_post), _ptr(w_pre), _ptr(gate), _ptr(r_out), 0, _ptr(dr_out),
                      _ptr(dh), _ptr(dr) if w_pre is not None else 0, _ptr(dy), _ptr(dw_post), _ptr(dw_pre),
                      _ptr(dgate))
    ws, n = _ws(moe_block_norm_workspace_size(args) if ws is None else 0, ws, device)
    moe_block_norm_backward(args, ws.data_ptr(), n, stream)
    return {"dr": dr, "dy": dy, "dw_post": dw_post, "dw_pre": dw_pre, "dgate": dgate}


def block_norm_backward(dr_out, dh, r_out, y=None, w_post=None, w_pre=None, gate=None, scale: float = 1.0,
                        eps: float = 1e-6, weight_offset: float = 0.0, ws=None, stream=None) -> dict:
    """Gradients of ``block_norm``, from its stored r_out and its inputs.

    dr_out [T, H] (None: zero; needed where there is no w_pre), dh [T, H]
    (with w_pre).  Returns dr (dr_out itself where there is no w_pre), dy,
    dw_post, dw_pre [H] float32 and dgate ([T, 1] or [H] float32, or [T, H] in
    the rows' type); None for what is not there."""
    ref = dr_out if dr_out is not None else dh
    if ref is None:
        raise ValueError("neither dr_out nor dh: nothing to compute")
    return _on(ref, stream, _block_norm_backward, dr_out, dh, r_out, y, w_post, w_pre, gate, scale, eps,
               weight_offset, ws)


# ---------------------------------------------------------------- embed
def _ids(ids, dev):
    if ids.dtype not in (torch.int64, torch.int32) or ids.dim() != 1 or ids.get_device() != dev:
        raise ValueError(f"ids: [T] int32 or int64 on device {dev} expected, got {ids.dtype} {list(ids.shape)}")
    return ids if ids.is_contiguous() else ids.contiguous()


def _embed(stream, table, ids, scale, out_dtype):
    V, H = table.shape
    code = _row_type(table.dtype, "table")
    out_dtype = table.dtype if out_dtype is None else out_dtype
    ocode = _same_or_f32(table.dtype, out_dtype, "out_dtype")
    ids = _ids(ids, table.get_device())
    T = ids.shape[0]
    table, ld = _rows(table, V, H, table.dtype, table.get_device(), "table")
    out = torch.empty((T, H), dtype=out_dtype, device=table.device)
    moe_embed(_EMBED.pack(T, H, V, code, ocode, ids.dtype is torch.int64, scale, 0, -1, ld, 0, ids.data_ptr(),
                          table.data_ptr(), out.data_ptr(), 0, 0), stream)
    return out


def embed(table, ids, scale: float = 1.0, out_dtype=None, stream=None):
    """out[t] = scale * table[ids[t]]: table [V, H], ids [T] int32 or int64;
    ``out_dtype``: the table's type (default) or float32.  An id outside the
    table gives a row of zeros and device status 5."""
    return _on(table, stream, _embed, table, ids, scale, out_dtype)


def _embed_backward(stream, ids, dout, V, scale, padding_id, dtable, ws):
    T, H = dout.shape
    code = _row_type(dout.dtype, "dout")
    dev = dout.get_device()
    ids = _ids(ids, dev)
    dout, ld = _rows(dout, ids.shape[0], H, dout.dtype, dev, "dout")
    accumulate = dtable is not None  # (into the caller's)
    if accumulate:
        if dtable.dtype is not torch.float32 or dtable.shape != (V, H) or not dtable.is_contiguous() or \
                dtable.get_device() != dev:
            raise ValueError(f"dtable: contiguous float32 [{V}, {H}] on device {dev} expected")
    else:
        dtable = torch.empty((V, H), dtype=torch.float32, device=dout.device)
    args = _EMBED.pack(T, H, V, code, code, ids.dtype is torch.int64, scale, accumulate,
                       -1 if padding_id is None else padding_id, 0, ld, ids.data_ptr(), 0, 0, dout.data_ptr(),
                       dtable.data_ptr())
    ws, n = _ws(moe_embed_workspace_size(args) if ws is None else 0, ws, dout.device)
    moe_embed_backward(args, ws.data_ptr(), n, stream)
    if accumulate:
        _written(dtable)
    return dtable


def embed_backward(ids, dout, num_embeddings: int, scale: float = 1.0, padding_id=None, dtable=None, ws=None,
                   stream=None):
    """The table's gradient, float32 [num_embeddings, H]: row v sums
    scale * dout[t] over the t with ids[t] = v, in ascending t.  ``dtable``:
    add to this tensor (only its rows that are hit are touched) instead of
    returning a new one; ``padding_id``: a token without gradient (one that is
    not in the table, -1 say: none)."""
    return _on(dout, stream, _embed_backward, ids, dout, num_embeddings, scale, padding_id, dtable, ws)


# ---------------------------------------------------------------- distill
def _teacher(logits, t_ids, t_logits, t_lse):
    T, V = logits.shape
    dev = logits.get_device()
    if t_ids.dim() != 2:
        raise ValueError("t_ids: [T, K] expected")
    K = t_ids.shape[1]
    t_ids, ld = _rows(t_ids, T, K, torch.int32, dev, "t_ids")
    t_logits, ld2 = _rows(t_logits, T, K, torch.float32, dev, "t_logits")
    if t_lse is not None:
        t_lse = _vec(t_lse, T, (torch.float32,), dev, "t_lse")
    return K, t_ids.contiguous() if ld else t_ids, t_logits.contiguous() if ld2 else t_logits, t_lse


def _distill(stream, logits, t_ids, t_logits, temperature, scale, t_lse, weight, lse, out, mode):
    T, V = logits.shape
    code, dev = _row_type(logits.dtype, "logits"), logits.get_device()
    K, t_ids, t_logits, t_lse = _teacher(logits, t_ids, t_logits, t_lse)
    given = logits
    logits, ld = _rows(logits, T, V, logits.dtype, dev, "logits")
    loss, ld_out, theirs = None, 0, out is not None
    if mode & 1:
        loss = torch.empty(T, dtype=torch.float32, device=logits.device)
    if mode == 1:
        lse = torch.empty(T, dtype=torch.float32, device=logits.device)
    elif mode == 2:
        lse = _vec(lse, T, (torch.float32,), dev, "lse")
    if mode & 2:
        weight = _vec(weight, T, (torch.float32,), dev, "weight")
        if out is None:
            out = _like(logits, ld)
        else:
            o, ld_out = _rows(out, T, V, logits.dtype, dev, "out")
            if o is not out or (out is given and logits is not given):
                raise ValueError("out: rows that cannot be written in place")
    args = _DISTILL.pack(T, V, K, code, temperature, scale, ld, ld_out, logits.data_ptr(), t_ids.data_ptr(),
                         t_logits.data_ptr(), _ptr(t_lse), _ptr(weight), _ptr(loss), _ptr(lse), _ptr(out))
    if mode == 1:
        moe_distill(args, stream)
        return loss, lse
    (moe_distill_backward if mode == 2 else moe_distill_step)(args, stream)
    if theirs:
        _written(out)
    return out if mode == 2 else (loss, out)


def distill(logits, t_ids, t_logits, temperature: float = 1.0, scale: float = 1.0, t_lse=None, stream=None):
    """(loss [T], lse [T]) float32 of the student's logits [T, V] against a
    teacher known by K tokens a row, t_ids [T, K] int32 (-1: no such slot) and
    t_logits [T, K] float32:

        loss_t = scale * sum_k p_k (log p_k - log softmax(logits_t / temperature)[id_k])

    p is the softmax of t_logits / temperature over the slots, or, with t_lse
    [T] (the teacher's log-sum-exp over its whole vocabulary at this
    temperature), exp(t_logits / temperature - t_lse)."""
    return _on(logits, stream, _distill, logits, t_ids, t_logits, temperature, scale, t_lse, None, None, None, 1)


def distill_backward(weight, lse, logits, t_ids, t_logits, temperature: float = 1.0, scale: float = 1.0, t_lse=None,
                     out=None, stream=None):
    """dlogits of ``distill`` for upstream gradients ``weight`` [T] float32 and
    the forward's lse, whose 24 bits bound what is known of the softmax (not
    for rows of nothing but the type's lowest value; ``distill_step`` takes
    them).  ``out``: written there (it may be ``logits`` itself)."""
    return _on(logits, stream, _distill, logits, t_ids, t_logits, temperature, scale, t_lse, weight, lse, out, 2)


def distill_step(logits, t_ids, t_logits, weight, temperature: float = 1.0, scale: float = 1.0, t_lse=None, out=None,
                 stream=None):
    """(loss, dlogits) in one pass: ``distill`` and ``distill_backward`` where
    the upstream gradient of each row's loss is known beforehand."""
    return _on(logits, stream, _distill, logits, t_ids, t_logits, temperature, scale, t_lse, weight, None, out, 3)
