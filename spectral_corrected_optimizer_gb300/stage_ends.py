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
come from torch's caching allocator on the current stream; a call given another
`stream` marks them as used there.
"""
from __future__ import annotations

from typing import NamedTuple

from . import _check, _ptr, _stream, _torch, lib

CKPT_GROUP = 128
_BF16, _FP32 = 0, 1


class NormCheckpoint(NamedTuple):
    """What residual_norm keeps for the backward pass: e4m3 values [rows, dim],
    fp32 scales [rows, ceil(dim / 128)], reciprocal root mean squares [rows]."""
    q: object
    scale: object
    rstd: object


def _type(t, name):
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return _BF16
    if t.dtype == torch.float32:
        return _FP32
    raise ValueError("%s must be bfloat16 or float32, got %s" % (name, t.dtype))


def _dtype(d, name):
    torch = _torch()
    if d not in (torch.bfloat16, torch.float32):
        raise ValueError("%s must be torch.bfloat16 or torch.float32, got %s" % (name, d))
    return d


def _matrix(t, shape, name, dtype=None):
    """Device pointer of a contiguous CUDA tensor of the given shape and dtype."""
    if tuple(t.shape) != tuple(shape) or (dtype is not None and t.dtype != dtype):
        raise ValueError("%s must be %sof shape %s, got %s %s" % (
            name, "" if dtype is None else "%s " % dtype, tuple(shape), t.dtype, tuple(t.shape)))
    return _ptr(t)


def _ids(t, name):
    torch = _torch()
    if t.dtype not in (torch.int32, torch.int64):
        raise ValueError("%s must be int32 or int64, got %s" % (name, t.dtype))
    return _ptr(t), t.element_size()


def _same_device(*tensors):
    devices = {t.device for t in tensors if t is not None}
    if len(devices) > 1:
        raise ValueError("tensors must be on one device, got %s" % sorted(map(str, devices)))


def _used_on(stream, *tensors):
    """The allocator must not hand these out again before `stream` is done with them."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _workspace(nbytes, device, what):
    torch = _torch()
    if nbytes < 0:
        raise ValueError("%s: %s" % (what, lib().specoptim_last_error().decode(errors="replace")))
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def _new(shape, dtype, device, stream):
    t = _torch().empty(shape, dtype=dtype, device=device)
    _used_on(stream, t)
    return t


# ---------------------------------------------------------------- embedding

def embed_lookup(table, ids, scale: float = 1.0, dtype=None, out=None, stream=None):
    """out[..., :] = scale * table[ids], rounded once to `dtype` (the table's by default).

    table: [vocab, dim] bf16 or fp32; ids: int32 or int64 of any shape.  The row
    of an id outside [0, vocab) is zero and check_device() reports it."""
    vocab, dim = table.shape
    dtype = _dtype(dtype or (table.dtype if out is None else out.dtype), "dtype")
    _same_device(table, ids, out)
    idp, idb = _ids(ids, "ids")
    tt, tp = _type(table, "table"), _ptr(table)
    shape = (*ids.shape, dim)
    if out is None:
        out = _new(shape, dtype, table.device, stream)
    op = _matrix(out, shape, "out", dtype)
    _check(lib().embed_lookup(tp, tt, idp, idb, ids.numel(), vocab, dim, float(scale), op, _type(out, "out"),
                              _stream(stream)), "embed_lookup")
    return out


def embed_grad(ids, dy, vocab: int, scale: float = 1.0, dtype=None, padding_idx: int | None = None, out=None,
               accumulate: bool = False, stream=None):
    """Gradient of embed_lookup: out[v] = scale * sum of dy over the tokens with id v (fp32 sums in token order).

    dy: [*ids.shape, dim] bf16 or fp32.  The result is dense [vocab, dim] in
    `dtype` (fp32 by default, what adamw takes); with accumulate=True it is added
    to `out`.  Tokens with id padding_idx contribute nothing."""
    torch = _torch()
    dim = dy.shape[-1]
    if accumulate and out is None:
        raise ValueError("accumulate=True needs the gradient to add to (out)")
    dtype = _dtype(dtype or (torch.float32 if out is None else out.dtype), "dtype")
    _same_device(ids, dy, out)
    idp, idb = _ids(ids, "ids")
    dp = _matrix(dy, (*ids.shape, dim), "dy")
    dt = _type(dy, "dy")
    if out is None:
        out = _new((vocab, dim), dtype, dy.device, stream)
    op = _matrix(out, (vocab, dim), "out", dtype)
    tokens = ids.numel()
    ws = _workspace(lib().embed_grad_workspace(tokens, vocab, dim), dy.device, "embed_grad")
    _used_on(stream, ws)
    _check(lib().embed_grad(idp, idb, dp, dt, tokens, vocab, dim, -1 if padding_idx is None else int(padding_idx),
                            float(scale), op, _type(out, "out"), int(accumulate), _ptr(ws), ws.numel(),
                            _stream(stream)), "embed_grad")
    return out


# ---------------------------------------------------------------- residual norm with an 8-bit checkpoint

def residual_norm(x, residual, gamma, eps: float = 1e-5, stream=None):
    """(checkpoint, s, y): s = x + residual, y = RMSNorm(s) * gamma, and s in 8 bits for the backward pass.

    x, residual: [rows, dim] bf16 or fp32 (residual None: s is x itself); gamma: [dim] of the same type."""
    torch = _torch()
    rows, dim = x.shape
    _same_device(x, residual, gamma)
    tp = _type(x, "x")
    xp = _ptr(x)
    rp = None if residual is None else _matrix(residual, (rows, dim), "residual", x.dtype)
    gp = _matrix(gamma, (dim,), "gamma", x.dtype)
    s = x if residual is None else _new((rows, dim), x.dtype, x.device, stream)
    y = _new((rows, dim), x.dtype, x.device, stream)
    kept = NormCheckpoint(_new((rows, dim), torch.float8_e4m3fn, x.device, stream),
                          _new((rows, -(-dim // CKPT_GROUP)), torch.float32, x.device, stream),
                          _new((rows,), torch.float32, x.device, stream))
    _check(lib().resnorm_forward(xp, rp, gp, tp, float(eps), _ptr(s), _ptr(y), _ptr(kept.q), _ptr(kept.scale),
                                 _ptr(kept.rstd), rows, dim, _stream(stream)), "resnorm_forward")
    return kept, s, y


def _kept(kept, rows, dim):
    torch = _torch()
    return (_matrix(kept.q, (rows, dim), "checkpoint values", torch.float8_e4m3fn),
            _matrix(kept.scale, (rows, -(-dim // CKPT_GROUP)), "checkpoint scales", torch.float32),
            _matrix(kept.rstd, (rows,), "checkpoint rstd", torch.float32))


def residual_norm_recompute(kept: NormCheckpoint, gamma, stream=None):
    """The norm's output once more, from its checkpoint (in gamma's type)."""
    rows, dim = kept.q.shape
    _same_device(kept.q, kept.scale, kept.rstd, gamma)
    qp, sp, rp = _kept(kept, rows, dim)
    gp = _matrix(gamma, (dim,), "gamma")
    tp = _type(gamma, "gamma")
    y = _new((rows, dim), gamma.dtype, gamma.device, stream)
    _check(lib().resnorm_recompute(qp, sp, rp, gp, tp, _ptr(y), rows, dim, _stream(stream)), "resnorm_recompute")
    return y


def residual_norm_backward(dy, kept: NormCheckpoint, gamma, ds=None, recompute: bool = False, stream=None):
    """(dx, dgamma, y) from dy = dL/dy and the checkpoint; dx is the gradient of both summands.

    ds: the gradient that reaches s through the residual stream (or None).
    dgamma is fp32.  y is the norm's recomputed output (recompute=True), else None."""
    torch = _torch()
    rows, dim = dy.shape
    _same_device(dy, ds, gamma, kept.q, kept.scale, kept.rstd)
    tp = _type(dy, "dy")
    dp = _ptr(dy)
    qp, sp, rp = _kept(kept, rows, dim)
    gp = _matrix(gamma, (dim,), "gamma", dy.dtype)
    dsp = None if ds is None else _matrix(ds, (rows, dim), "ds", dy.dtype)
    dx = _new((rows, dim), dy.dtype, dy.device, stream)
    dgamma = _new((dim,), torch.float32, dy.device, stream)
    y = _new((rows, dim), dy.dtype, dy.device, stream) if recompute else None
    ws = _workspace(lib().resnorm_backward_workspace(rows, dim), dy.device, "resnorm_backward")
    _used_on(stream, ws)
    _check(lib().resnorm_backward(dp, dsp, qp, sp, rp, gp, tp, _ptr(dx), _ptr(dgamma), _ptr(y), rows, dim, _ptr(ws),
                                  ws.numel(), _stream(stream)), "resnorm_backward")
    return dx, dgamma, y


# ---------------------------------------------------------------- vocabulary head

def _head_args(h, w, targets, reduction):
    torch = _torch()
    if reduction not in ("mean", "sum"):
        raise ValueError("reduction must be 'mean' or 'sum', got %r" % (reduction,))
    tokens, dim = h.shape
    vocab = w.shape[0]
    _same_device(h, w, targets)
    hp = _matrix(h, (tokens, dim), "h", torch.bfloat16)
    wp = _matrix(w, (vocab, dim), "w", torch.bfloat16)
    tp, tb = _ids(targets, "targets")
    if tuple(targets.shape) != (tokens,):
        raise ValueError("targets must have shape (%d,), got %s" % (tokens, tuple(targets.shape)))
    return tokens, vocab, dim, hp, wp, tp, tb, int(reduction == "mean")


def head_loss(h, w, targets, ignore_index: int = -100, reduction: str = "mean", stream=None):
    """(loss, row_loss): softmax cross entropy of h @ w.T against targets, without the logits in memory.

    h: [tokens, dim] bf16, w: [vocab, dim] bf16, targets: [tokens] int32 or int64.
    Tokens with target ignore_index have row_loss 0 and do not count in the mean."""
    torch = _torch()
    tokens, vocab, dim, hp, wp, tp, tb, mean = _head_args(h, w, targets, reduction)
    loss = _new((), torch.float32, h.device, stream)
    row_loss = _new((tokens,), torch.float32, h.device, stream)
    ws = _workspace(lib().head_loss_workspace(tokens, vocab, dim), h.device, "head_loss")
    _used_on(stream, ws)
    _check(lib().head_loss(hp, wp, tp, tb, int(ignore_index), tokens, vocab, dim, mean, _ptr(loss), _ptr(row_loss),
                           _ptr(ws), ws.numel(), _stream(stream)), "head_loss")
    return loss, row_loss


def head_loss_grad(h, w, targets, ignore_index: int = -100, reduction: str = "mean", grad_scale: float = 1.0,
                   dtype=None, dw=None, accumulate: bool = False, stream=None):
    """(loss, row_loss, dh, dw): head_loss and the gradients of grad_scale * loss.

    dh is bf16.  dw is [vocab, dim] in `dtype` (fp32 by default, what adamw
    takes); with accumulate=True it is added to the given `dw`."""
    torch = _torch()
    tokens, vocab, dim, hp, wp, tp, tb, mean = _head_args(h, w, targets, reduction)
    if accumulate and dw is None:
        raise ValueError("accumulate=True needs the gradient to add to (dw)")
    dtype = _dtype(dtype or (torch.float32 if dw is None else dw.dtype), "dtype")
    _same_device(h, dw)
    if dw is None:
        dw = _new((vocab, dim), dtype, h.device, stream)
    dwp = _matrix(dw, (vocab, dim), "dw", dtype)
    loss = _new((), torch.float32, h.device, stream)
    row_loss = _new((tokens,), torch.float32, h.device, stream)
    dh = _new((tokens, dim), torch.bfloat16, h.device, stream)
    ws = _workspace(lib().head_loss_grad_workspace(tokens, vocab, dim), h.device, "head_loss_grad")
    _used_on(stream, ws)
    _check(lib().head_loss_grad(hp, wp, tp, tb, int(ignore_index), tokens, vocab, dim, mean, float(grad_scale),
                                _ptr(loss), _ptr(row_loss), _ptr(dh), dwp, _type(dw, "dw"), int(accumulate), _ptr(ws),
                                ws.numel(), _stream(stream)), "head_loss_grad")
    return loss, row_loss, dh, dw
