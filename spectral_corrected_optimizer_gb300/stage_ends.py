"""Binding of include/stage_ends.h (argument marshalling only): the operators of
a training pipeline's end stages, beside the masked boundary between them.

  embed_lookup, embed_grad              the first stage's embedding and its
                                        gradient by sorted tokens
  residual_norm, residual_norm_recompute, residual_norm_backward
                                        residual sum + RMSNorm whose input is
                                        kept in 8 bits for the backward pass
  head_loss, head_loss_grad             softmax cross entropy over a large
                                        vocabulary without keeping the logits,
                                        and its gradients

Every operation runs in the library's CUDA kernels.  Outputs and workspaces
come from torch's caching allocator.  With `stream` given, a call allocates and
runs on that stream and marks its inputs as used there; waiting for the inputs
and for the outputs is the caller's, as with any work on two streams.  Tensors
are on the current device; calls on another one's are refused.
"""
from __future__ import annotations

from typing import NamedTuple

import torch

from . import _check, lib

CKPT_GROUP = 128
_BF16, _FP32 = 0, 1
_TYPES = {torch.bfloat16: _BF16, torch.float32: _FP32}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


class NormCheckpoint(NamedTuple):
    """What residual_norm keeps for the backward pass: e4m3 values [rows, dim],
    fp32 scales [rows, ceil(dim / 128)], reciprocal root mean squares [rows]."""
    q: torch.Tensor
    scale: torch.Tensor
    rstd: torch.Tensor


# The small calls are as long as their marshalling, so each argument costs one
# plain test; the messages are put together only when one fails.

def _type(dtype, name):
    code = _TYPES.get(dtype)
    if code is None:
        raise ValueError("%s must be bfloat16 or float32, got %s" % (name, dtype))
    return code


def _ids(t, device, name):
    width = _ID_BYTES.get(t.dtype)
    if width is None:
        raise ValueError("%s must be int32 or int64, got %s" % (name, t.dtype))
    return _ptr(t, device, name), width


def _ptr(t, device, name):
    """Device pointer of a contiguous tensor on the call's device."""
    if not t.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _matrix(t, shape, dtype, device, name):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError("%s must be %s of shape %s, got %s %s" % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))
    return _ptr(t, device, name)


def _stream(device):
    """The current stream of the call's device, which has to be the current one: kernels are launched there."""
    if device.index != torch._C._cuda_getDevice():
        raise ValueError("tensors are on %s, the current device is cuda:%d" % (device, torch._C._cuda_getDevice()))
    return torch._C._cuda_getCurrentRawStream(device.index)


def _workspace(nbytes, device, what):
    if nbytes < 0:
        raise ValueError("%s: %s" % (what, lib().specoptim_last_error().decode(errors="replace")))
    t = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    return t, t.data_ptr()


def _on(stream, call, *args, **kwargs):
    """The same call with `stream` current: what it allocates belongs to that stream, what it is given is in use there."""
    with torch.cuda.stream(stream):
        result = call(*args, **kwargs)
    for a in (*args, *kwargs.values()):
        for t in a if isinstance(a, NormCheckpoint) else (a,):
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)
    return result


# ---------------------------------------------------------------- embedding

def embed_lookup(table, ids, scale: float = 1.0, dtype=None, out=None, stream=None):
    """out[..., :] = scale * table[ids], rounded once to `dtype` (the table's by default).

    table: [vocab, dim] bf16 or fp32; ids: int32 or int64 of any shape.  The row
    of an id outside [0, vocab) is zero and check_device() reports it."""
    if stream is not None:
        return _on(stream, embed_lookup, table, ids, scale=scale, dtype=dtype, out=out)
    vocab, dim = table.shape
    device = table.device
    if dtype is None:
        dtype = table.dtype if out is None else out.dtype
    code = _type(dtype, "dtype")
    idp, idb = _ids(ids, device, "ids")
    tt, tp = _type(table.dtype, "table"), _ptr(table, device, "table")
    shape = (*ids.shape, dim)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    op = _matrix(out, shape, dtype, device, "out")
    _check(lib().embed_lookup(tp, tt, idp, idb, ids.numel(), vocab, dim, scale, op, code, _stream(device)),
           "embed_lookup")
    return out


def embed_grad(ids, dy, vocab: int, scale: float = 1.0, dtype=None, padding_idx: int | None = None, out=None,
               accumulate: bool = False, stream=None):
    """Gradient of embed_lookup: out[v] = scale * sum of dy over the tokens with id v (fp32 sums in token order).

    dy: [*ids.shape, dim] bf16 or fp32.  The result is dense [vocab, dim] in
    `dtype` (fp32 by default, what adamw takes); with accumulate=True it is added
    to `out`.  Tokens with id padding_idx contribute nothing."""
    if stream is not None:
        return _on(stream, embed_grad, ids, dy, vocab, scale=scale, dtype=dtype, padding_idx=padding_idx, out=out,
                   accumulate=accumulate)
    dim = dy.shape[-1]
    device = dy.device
    if accumulate and out is None:
        raise ValueError("accumulate=True needs the gradient to add to (out)")
    if dtype is None:
        dtype = torch.float32 if out is None else out.dtype
    code, dt = _type(dtype, "dtype"), _type(dy.dtype, "dy")
    idp, idb = _ids(ids, device, "ids")
    dp = _matrix(dy, (*ids.shape, dim), dy.dtype, device, "dy")
    if out is None:
        out = torch.empty((vocab, dim), dtype=dtype, device=device)
    op = _matrix(out, (vocab, dim), dtype, device, "out")
    tokens = ids.numel()
    ws, wp = _workspace(lib().embed_grad_workspace(tokens, vocab, dim), device, "embed_grad")
    _check(lib().embed_grad(idp, idb, dp, dt, tokens, vocab, dim, -1 if padding_idx is None else padding_idx, scale,
                            op, code, accumulate, wp, ws.numel(), _stream(device)), "embed_grad")
    return out


# ---------------------------------------------------------------- residual norm with an 8-bit checkpoint

def residual_norm(x, residual, gamma, eps: float = 1e-5, stream=None):
    """(checkpoint, s, y): s = x + residual, y = RMSNorm(s) * gamma, and s in 8 bits for the backward pass.

    x, residual: [rows, dim] bf16 or fp32 (residual None: s is x itself); gamma: [dim] of the same type."""
    if stream is not None:
        return _on(stream, residual_norm, x, residual, gamma, eps)
    shape = x.shape
    rows, dim = shape
    device, dtype = x.device, x.dtype
    code = _type(dtype, "x")
    xp = _ptr(x, device, "x")
    gp = _matrix(gamma, (dim,), dtype, device, "gamma")
    if residual is None:
        rp, s, sp = None, x, None
    else:
        rp = _matrix(residual, shape, dtype, device, "residual")
        s = torch.empty_like(x)
        sp = s.data_ptr()
    y = torch.empty_like(x)
    kept = NormCheckpoint(torch.empty(shape, dtype=torch.float8_e4m3fn, device=device),
                          torch.empty((rows, (dim + CKPT_GROUP - 1) // CKPT_GROUP), dtype=torch.float32, device=device),
                          torch.empty(rows, dtype=torch.float32, device=device))
    _check(lib().resnorm_forward(xp, rp, gp, code, eps, sp, y.data_ptr(), kept.q.data_ptr(), kept.scale.data_ptr(),
                                 kept.rstd.data_ptr(), rows, dim, _stream(device)), "resnorm_forward")
    return kept, s, y


def _kept(kept, rows, dim, device):
    return (_matrix(kept.q, (rows, dim), torch.float8_e4m3fn, device, "checkpoint values"),
            _matrix(kept.scale, (rows, (dim + CKPT_GROUP - 1) // CKPT_GROUP), torch.float32, device,
                    "checkpoint scales"),
            _matrix(kept.rstd, (rows,), torch.float32, device, "checkpoint rstd"))


def residual_norm_recompute(kept: NormCheckpoint, gamma, stream=None):
    """The norm's output once more, from its checkpoint (in gamma's type)."""
    if stream is not None:
        return _on(stream, residual_norm_recompute, kept, gamma)
    rows, dim = kept.q.shape
    device = gamma.device
    qp, sp, rp = _kept(kept, rows, dim, device)
    code = _type(gamma.dtype, "gamma")
    gp = _matrix(gamma, (dim,), gamma.dtype, device, "gamma")
    y = torch.empty((rows, dim), dtype=gamma.dtype, device=device)
    _check(lib().resnorm_recompute(qp, sp, rp, gp, code, y.data_ptr(), rows, dim, _stream(device)),
           "resnorm_recompute")
    return y


def residual_norm_backward(dy, kept: NormCheckpoint, gamma, ds=None, recompute: bool = False, stream=None):
    """(dx, dgamma, y) from dy = dL/dy and the checkpoint; dx is the gradient of both summands.

    ds: the gradient that reaches s through the residual stream (or None).
    dgamma is fp32.  y is the norm's recomputed output (recompute=True), else None."""
    if stream is not None:
        return _on(stream, residual_norm_backward, dy, kept, gamma, ds=ds, recompute=recompute)
    shape = dy.shape
    rows, dim = shape
    device, dtype = dy.device, dy.dtype
    code = _type(dtype, "dy")
    dp = _ptr(dy, device, "dy")
    qp, sp, rp = _kept(kept, rows, dim, device)
    gp = _matrix(gamma, (dim,), dtype, device, "gamma")
    dsp = None if ds is None else _matrix(ds, shape, dtype, device, "ds")
    dx = torch.empty_like(dy)
    dgamma = torch.empty(dim, dtype=torch.float32, device=device)
    y = torch.empty_like(dy) if recompute else None
    ws, wp = _workspace(lib().resnorm_backward_workspace(rows, dim), device, "resnorm_backward")
    _check(lib().resnorm_backward(dp, dsp, qp, sp, rp, gp, code, dx.data_ptr(), dgamma.data_ptr(),
                                  y.data_ptr() if recompute else None, rows, dim, wp, ws.numel(), _stream(device)),
           "resnorm_backward")
    return dx, dgamma, y


# ---------------------------------------------------------------- vocabulary head

def _head_args(h, w, targets, reduction):
    if reduction not in ("mean", "sum"):
        raise ValueError("reduction must be 'mean' or 'sum', got %r" % (reduction,))
    tokens, dim = h.shape
    vocab = w.shape[0]
    device = h.device
    hp = _matrix(h, (tokens, dim), torch.bfloat16, device, "h")
    wp = _matrix(w, (vocab, dim), torch.bfloat16, device, "w")
    tp, tb = _ids(targets, device, "targets")
    if targets.shape != (tokens,):
        raise ValueError("targets must have shape (%d,), got %s" % (tokens, tuple(targets.shape)))
    return tokens, vocab, dim, device, hp, wp, tp, tb, reduction == "mean"


def head_loss(h, w, targets, ignore_index: int = -100, reduction: str = "mean", stream=None):
    """(loss, row_loss): softmax cross entropy of h @ w.T against targets, without the logits in memory.

    h: [tokens, dim] bf16, w: [vocab, dim] bf16 (16-byte aligned), targets: [tokens] int32 or int64.
    Tokens with target ignore_index have row_loss 0 and do not count in the mean."""
    if stream is not None:
        return _on(stream, head_loss, h, w, targets, ignore_index=ignore_index, reduction=reduction)
    tokens, vocab, dim, device, hp, wp, tp, tb, mean = _head_args(h, w, targets, reduction)
    loss = torch.empty((), dtype=torch.float32, device=device)
    row_loss = torch.empty(tokens, dtype=torch.float32, device=device)
    ws, wsp = _workspace(lib().head_loss_workspace(tokens, vocab, dim), device, "head_loss")
    _check(lib().head_loss(hp, wp, tp, tb, ignore_index, tokens, vocab, dim, mean, loss.data_ptr(),
                           row_loss.data_ptr(), wsp, ws.numel(), _stream(device)), "head_loss")
    return loss, row_loss


def head_loss_grad(h, w, targets, ignore_index: int = -100, reduction: str = "mean", grad_scale: float = 1.0,
                   dtype=None, dw=None, accumulate: bool = False, stream=None):
    """(loss, row_loss, dh, dw): head_loss and the gradients of grad_scale * loss.

    dh is bf16.  dw is [vocab, dim] in `dtype` (fp32 by default, what adamw
    takes); with accumulate=True it is added to the given `dw`.  Probabilities
    are rounded to bf16 whatever `dtype` is.  Some forms store dw value by value
    and are slow where tokens are few: a bf16 dw that is added to, and any dw
    that is not 16-byte aligned or whose rows are not multiples of 16 bytes
    (2048 tokens, 128256 x 2048: 2.3 ms, bf16 added 8.1 ms).  A width that is no
    multiple of 8 also costs a padded copy of w in every call (0.3 ms there)."""
    if stream is not None:
        return _on(stream, head_loss_grad, h, w, targets, ignore_index=ignore_index, reduction=reduction,
                   grad_scale=grad_scale, dtype=dtype, dw=dw, accumulate=accumulate)
    if accumulate and dw is None:
        raise ValueError("accumulate=True needs the gradient to add to (dw)")
    tokens, vocab, dim, device, hp, wp, tp, tb, mean = _head_args(h, w, targets, reduction)
    if dtype is None:
        dtype = torch.float32 if dw is None else dw.dtype
    code = _type(dtype, "dtype")
    if dw is None:
        dw = torch.empty((vocab, dim), dtype=dtype, device=device)
    dwp = _matrix(dw, (vocab, dim), dtype, device, "dw")
    loss = torch.empty((), dtype=torch.float32, device=device)
    row_loss = torch.empty(tokens, dtype=torch.float32, device=device)
    dh = torch.empty_like(h)
    ws, wsp = _workspace(lib().head_loss_grad_workspace(tokens, vocab, dim), device, "head_loss_grad")
    _check(lib().head_loss_grad(hp, wp, tp, tb, ignore_index, tokens, vocab, dim, mean, grad_scale,
                                loss.data_ptr(), row_loss.data_ptr(), dh.data_ptr(), dwp, code, accumulate, wsp,
                                ws.numel(), _stream(device)), "head_loss_grad")
    return loss, row_loss, dh, dw
