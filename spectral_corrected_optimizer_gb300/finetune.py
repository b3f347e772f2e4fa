"""Binding of include/finetune.h (argument marshalling only): the operators of a
fine-tuning step, beside the end stages' (``stage_ends``) and the optimizer's.

  layer_norm, layer_norm_backward       residual sum + LayerNorm and its
                                        gradients
  head_logp, head_logp_backward         log-probabilities of given tokens under
                                        the vocabulary head, and the gradient of
                                        any loss over them
  preference_loss                       loss over pairs of sequences
  policy_loss                           clipped policy ratio with a KL term
  grad_norm, clip_grads                 global norm and clipping of all gradients

The losses return their gradient with respect to the log-probabilities, which
head_logp_backward takes.  Every operation runs in the library's CUDA kernels.
Outputs and workspaces come from torch's caching allocator.  With `stream`
given, a call allocates and runs on that stream and marks its inputs as used
there; waiting for the inputs and for the outputs is the caller's.  Tensors are on
the current device; calls on another one's are refused.
"""
from __future__ import annotations

import math
from array import array
from typing import NamedTuple

import torch

from . import _check, lib
from .stage_ends import _ID_BYTES, _ids, _matrix, _ptr, _stream, _type, _TYPES, _workspace

_KINDS = {"logistic": 0, "hinge": 1, "square": 2}
_REDUCTIONS = {"token": 0, "sequence": 1, "sum": 2}
_NORMS = {2: 0, math.inf: 1}
_MASKS = (torch.bool, torch.uint8)


class NormStatistics(NamedTuple):
    """What layer_norm keeps of each row beside s: its mean and the reciprocal standard deviation, fp32 [rows]."""
    mean: torch.Tensor
    rstd: torch.Tensor


def _record(a, stream):
    if isinstance(a, torch.Tensor):
        if a.is_cuda:
            a.record_stream(stream)
    elif isinstance(a, (list, tuple)):
        for x in a:
            _record(x, stream)


def _on(stream, call, *args, **kwargs):
    """The same call with `stream` current: what it allocates belongs to that stream, what it is given is in use there."""
    with torch.cuda.stream(stream):
        result = call(*args, **kwargs)
    _record([*args, *kwargs.values()], stream)
    return result


# ---------------------------------------------------------------- layer norm

def layer_norm(x, residual, gamma, beta=None, eps: float = 1e-5, stream=None):
    """(statistics, s, y): s = x + residual, y = (s - mean) * rstd * gamma + beta.

    x, residual: [rows, dim] bf16 or fp32 (residual None: s is x itself); gamma, beta: [dim] of the same type (beta
    None: none)."""
    if stream is not None:
        return _on(stream, layer_norm, x, residual, gamma, beta, eps)
    shape = x.shape
    rows, dim = shape
    device, dtype = x.device, x.dtype
    code = _type(dtype, "x")
    xp = _ptr(x, device, "x")
    gp = _matrix(gamma, (dim,), dtype, device, "gamma")
    bp = None if beta is None else _matrix(beta, (dim,), dtype, device, "beta")
    if residual is None:
        rp, s, sp = None, x, None
    else:
        rp = _matrix(residual, shape, dtype, device, "residual")
        s = torch.empty_like(x)
        sp = s.data_ptr()
    y = torch.empty_like(x)
    kept = NormStatistics(torch.empty(rows, dtype=torch.float32, device=device),
                          torch.empty(rows, dtype=torch.float32, device=device))
    _check(lib().layernorm_forward(xp, rp, gp, bp, code, eps, sp, y.data_ptr(), kept.mean.data_ptr(),
                                   kept.rstd.data_ptr(), rows, dim, _stream(device)), "layernorm_forward")
    return kept, s, y


def layer_norm_backward(dy, s, kept: NormStatistics, gamma, ds=None, bias: bool = True, stream=None):
    """(dx, dgamma, dbeta) from dy = dL/dy and what the forward pass gave; dx is the gradient of both summands.

    ds: the gradient that reaches s through the residual stream (or None).  dgamma and dbeta are fp32, what adamw takes;
    dbeta is None with bias=False."""
    if stream is not None:
        return _on(stream, layer_norm_backward, dy, s, kept, gamma, ds=ds, bias=bias)
    shape = dy.shape
    rows, dim = shape
    device, dtype = dy.device, dy.dtype
    code = _type(dtype, "dy")
    dp = _ptr(dy, device, "dy")
    sp = _matrix(s, shape, dtype, device, "s")
    mp = _matrix(kept.mean, (rows,), torch.float32, device, "mean")
    rp = _matrix(kept.rstd, (rows,), torch.float32, device, "rstd")
    gp = _matrix(gamma, (dim,), dtype, device, "gamma")
    dsp = None if ds is None else _matrix(ds, shape, dtype, device, "ds")
    dx = torch.empty_like(dy)
    dgamma = torch.empty(dim, dtype=torch.float32, device=device)
    dbeta = torch.empty(dim, dtype=torch.float32, device=device) if bias else None
    ws, wp = _workspace(lib().layernorm_backward_workspace(rows, dim), device, "layernorm_backward")
    _check(lib().layernorm_backward(dp, dsp, sp, mp, rp, gp, code, dx.data_ptr(), dgamma.data_ptr(),
                                    dbeta.data_ptr() if bias else None, rows, dim, wp, ws.numel(), _stream(device)),
           "layernorm_backward")
    return dx, dgamma, dbeta


# ---------------------------------------------------------------- log-probabilities under the head

def _head_args(h, w, targets):
    tokens, dim = h.shape
    vocab = w.shape[0]
    device = h.device
    hp = _matrix(h, (tokens, dim), torch.bfloat16, device, "h")
    wp = _matrix(w, (vocab, dim), torch.bfloat16, device, "w")
    tp, tb = _ids(targets, device, "targets")
    if targets.shape != (tokens,):
        raise ValueError("targets must have shape (%d,), got %s" % (tokens, tuple(targets.shape)))
    return tokens, vocab, dim, device, hp, wp, tp, tb


def head_logp(h, w, targets, ignore_index: int = -100, stream=None):
    """(logp, kept): log-probabilities [tokens] of the targets under softmax(h @ w.T), without the logits in memory.

    h: [tokens, dim] bf16, w: [vocab, dim] bf16 (16-byte aligned), targets: [tokens] int32 or int64.  Tokens with target
    ignore_index have logp 0.  kept (fp32 [3, tokens]) is what head_logp_backward needs of the forward pass."""
    if stream is not None:
        return _on(stream, head_logp, h, w, targets, ignore_index=ignore_index)
    tokens, vocab, dim, device, hp, wp, tp, tb = _head_args(h, w, targets)
    logp = torch.empty(tokens, dtype=torch.float32, device=device)
    kept = torch.empty((3, tokens), dtype=torch.float32, device=device)
    ws, wsp = _workspace(lib().head_logp_workspace(tokens, vocab, dim), device, "head_logp")
    _check(lib().head_logp(hp, wp, tp, tb, ignore_index, tokens, vocab, dim, logp.data_ptr(), kept.data_ptr(), wsp,
                           ws.numel(), _stream(device)), "head_logp")
    return logp, kept


def head_logp_backward(dlogp, kept, h, w, targets, ignore_index: int = -100, dtype=None, dw=None,
                       accumulate: bool = False, stream=None):
    """(dh, dw) of a loss with gradient dlogp [tokens] (fp32) in the log-probabilities that head_logp gave.

    dh is bf16.  dw is [vocab, dim] in `dtype` (fp32 by default, what adamw takes); with accumulate=True it is added to
    the given `dw`.  Tokens whose dlogp is 0 cost nothing.  What head_loss_grad says of slow forms of dw holds here."""
    if stream is not None:
        return _on(stream, head_logp_backward, dlogp, kept, h, w, targets, ignore_index=ignore_index, dtype=dtype, dw=dw,
                   accumulate=accumulate)
    if accumulate and dw is None:
        raise ValueError("accumulate=True needs the gradient to add to (dw)")
    tokens, vocab, dim, device, hp, wp, tp, tb = _head_args(h, w, targets)
    gp = _matrix(dlogp, (tokens,), torch.float32, device, "dlogp")
    kp = _matrix(kept, (3, tokens), torch.float32, device, "kept")
    if dtype is None:
        dtype = torch.float32 if dw is None else dw.dtype
    code = _type(dtype, "dtype")
    if dw is None:
        dw = torch.empty((vocab, dim), dtype=dtype, device=device)
    dwp = _matrix(dw, (vocab, dim), dtype, device, "dw")
    dh = torch.empty_like(h)
    ws, wsp = _workspace(lib().head_logp_backward_workspace(tokens, vocab, dim), device, "head_logp_backward")
    _check(lib().head_logp_backward(gp, kp, hp, wp, tp, tb, ignore_index, tokens, vocab, dim, dh.data_ptr(), dwp, code,
                                    accumulate, wsp, ws.numel(), _stream(device)), "head_logp_backward")
    return dh, dw


# ---------------------------------------------------------------- losses over log-probabilities

def _room(nbytes, device, what):
    """Workspace, its pointer and its size; small calls need none."""
    if nbytes == 0:
        return None, None, 0
    ws, pointer = _workspace(nbytes, device, what)
    return ws, pointer, ws.numel()


def _per_token(t, tokens, device, name):
    return None if t is None else _matrix(t, (tokens,), torch.float32, device, name)


def _mask(mask, tokens, device):
    if mask is None:
        return None
    if mask.dtype not in _MASKS or mask.shape != (tokens,):
        raise ValueError("mask must be bool or uint8 of shape (%d,), got %s %s" % (tokens, mask.dtype, tuple(mask.shape)))
    return _ptr(mask, device, "mask")


def _offsets(offsets, device):
    width = _ID_BYTES.get(offsets.dtype)
    if width is None or offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("offsets must be int32 or int64 with one value more than sequences, got %s %s"
                         % (offsets.dtype, tuple(offsets.shape)))
    return _ptr(offsets, device, "offsets"), width, offsets.numel() - 1


def preference_loss(logp, ref_logp, offsets, beta: float = 0.1, kind: str = "logistic", smoothing: float = 0.0,
                    average: bool = False, mask=None, reduction: str = "mean", grad_scale: float = 1.0, stream=None):
    """(loss, pair_loss, rewards, dlogp) of pairs of sequences: 2p is preferred to 2p + 1.

    logp, ref_logp: fp32 [tokens] (ref_logp None: 0), the sequences one behind the other; offsets: int32 or int64
    [2 * pairs + 1], where each begins and the last ends.  mask: bool or uint8 [tokens], the tokens that count.  A
    sequence's score is the sum (average=True: the mean) of logp - ref_logp over its tokens; rewards [pairs, 2] are beta
    times the scores, delta their difference.  kind: "logistic" (with label smoothing), "hinge" or "square".  dlogp is the
    gradient of grad_scale * loss, 0 at tokens that do not count."""
    if stream is not None:
        return _on(stream, preference_loss, logp, ref_logp, offsets, beta=beta, kind=kind, smoothing=smoothing,
                   average=average, mask=mask, reduction=reduction, grad_scale=grad_scale)
    code = _KINDS.get(kind)
    if code is None:
        raise ValueError("kind must be 'logistic', 'hinge' or 'square', got %r" % (kind,))
    if reduction not in ("mean", "sum"):
        raise ValueError("reduction must be 'mean' or 'sum', got %r" % (reduction,))
    tokens, device = logp.numel(), logp.device
    lp = _per_token(logp, tokens, device, "logp")
    rp = _per_token(ref_logp, tokens, device, "ref_logp")
    mp = _mask(mask, tokens, device)
    op, ob, count = _offsets(offsets, device)
    if count % 2:
        raise ValueError("offsets must be those of pairs of sequences: an odd number of values, got %d" % (count + 1))
    pairs = count // 2
    loss = torch.empty((), dtype=torch.float32, device=device)
    pair_loss = torch.empty(pairs, dtype=torch.float32, device=device)
    rewards = torch.empty((pairs, 2), dtype=torch.float32, device=device)
    dlogp = torch.empty(tokens, dtype=torch.float32, device=device)
    ws, wsp, wsn = _room(lib().preference_loss_workspace(pairs, tokens), device, "preference_loss")
    _check(lib().preference_loss(lp, rp, mp, op, ob, pairs, tokens, code, beta, smoothing, average, reduction == "mean",
                                 grad_scale, loss.data_ptr(), pair_loss.data_ptr(), rewards.data_ptr(),
                                 dlogp.data_ptr(), wsp, wsn, _stream(device)), "preference_loss")
    return loss, pair_loss, rewards, dlogp


def policy_loss(logp, old_logp, advantages, offsets=None, ref_logp=None, mask=None, clip_low: float = 0.2,
                clip_high: float = 0.2, kl_coef: float = 0.0, reduction: str = "token", grad_scale: float = 1.0,
                per_sequence: bool | None = None, stream=None):
    """(loss, parts, dlogp) of the clipped policy ratio exp(logp - old_logp) with a KL term against ref_logp.

    logp, old_logp, ref_logp: fp32 [tokens]; advantages: fp32 [tokens], or one per sequence ([sequences], which then needs
    offsets).  offsets: int32 or int64 [sequences + 1], where each sequence begins and the last ends (None: all tokens are
    one).  mask: bool or uint8 [tokens], the tokens that count.  reduction: "token" (mean over them), "sequence" (mean of
    the sequences' means) or "sum".  parts (fp32 [3]): the policy part of the loss, the KL divergence and the clipped share,
    aggregated alike; loss = parts[0] + kl_coef * parts[1] (with kl_coef 0 the divergence is only reported).  dlogp is the gradient of grad_scale * loss, 0 at tokens that
    do not count.  per_sequence says which advantages are given; it is needed only where tokens and sequences are as many."""
    if stream is not None:
        return _on(stream, policy_loss, logp, old_logp, advantages, offsets=offsets, ref_logp=ref_logp, mask=mask,
                   clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef, reduction=reduction, grad_scale=grad_scale,
                   per_sequence=per_sequence)
    code = _REDUCTIONS.get(reduction)
    if code is None:
        raise ValueError("reduction must be 'token', 'sequence' or 'sum', got %r" % (reduction,))
    tokens, device = logp.numel(), logp.device
    lp = _per_token(logp, tokens, device, "logp")
    dp = _per_token(old_logp, tokens, device, "old_logp")
    rp = _per_token(ref_logp, tokens, device, "ref_logp")
    if dp is None:
        raise ValueError("old_logp must be given")
    if ref_logp is None and kl_coef != 0:
        raise ValueError("kl_coef needs ref_logp")
    mp = _mask(mask, tokens, device)
    op, ob, count = (None, 8, 1) if offsets is None else _offsets(offsets, device)
    if per_sequence is None:
        per_sequence = advantages.shape != (tokens,)
        if not per_sequence and offsets is not None and count == tokens:
            raise ValueError("there are as many sequences as tokens: say with per_sequence which advantages these are")
    if per_sequence and offsets is None:
        raise ValueError("advantages must have shape (%d,) without offsets, got %s" % (tokens, tuple(advantages.shape)))
    ap = _matrix(advantages, (count,) if per_sequence else (tokens,), torch.float32, device, "advantages")
    loss = torch.empty((), dtype=torch.float32, device=device)
    parts = torch.empty(3, dtype=torch.float32, device=device)
    dlogp = torch.empty(tokens, dtype=torch.float32, device=device)
    ws, wsp, wsn = _room(lib().policy_loss_workspace(count, tokens), device, "policy_loss")
    _check(lib().policy_loss(lp, dp, rp, mp, ap, per_sequence, op, ob, count, tokens, clip_low, clip_high, kl_coef, code,
                             grad_scale, loss.data_ptr(), parts.data_ptr(), dlogp.data_ptr(), wsp, wsn, _stream(device)),
           "policy_loss")
    return loss, parts, dlogp


# ---------------------------------------------------------------- gradient norm and clipping

def _tensors(tensors, device, name):
    """Host arrays of the tensors' pointers, sizes and types (kept alive by the caller), and the number of them."""
    types = [_TYPES.get(t.dtype) for t in tensors]
    for t, code in zip(tensors, types):
        if code is None or t.device != device or not t.is_contiguous():
            _type(t.dtype, name)
            _ptr(t, device, name)
    return array("Q", [t.data_ptr() for t in tensors]), array("q", [t.numel() for t in tensors]), array("i", types)


def _address(a):
    return a.buffer_info()[0]


def _norm_kind(norm_type):
    kind = _NORMS.get(norm_type)
    if kind is None:
        raise ValueError("norm_type must be 2 or inf, got %r" % (norm_type,))
    return kind


def _device_of(grads):
    if not grads:
        return torch.device("cuda", torch.cuda.current_device())
    if not grads[0].is_cuda:
        raise ValueError("grads must be on a CUDA device")
    return grads[0].device


def grad_norm(grads, scale: float = 1.0, norm_type: float = 2.0, stream=None):
    """Norm (a fp32 scalar) of scale * g over the values of all tensors together, norm_type 2 or inf.

    grads: contiguous CUDA tensors, bf16 or fp32 each."""
    grads = list(grads)
    if stream is not None:
        return _on(stream, grad_norm, grads, scale=scale, norm_type=norm_type)
    kind = _norm_kind(norm_type)
    device = _device_of(grads)
    pointers, sizes, types = _tensors(grads, device, "grads")
    norm = torch.empty((), dtype=torch.float32, device=device)
    ws, wsp = _workspace(lib().grad_norm_workspace(len(grads)), device, "grad_norm")
    _check(lib().grad_norm(_address(pointers), _address(sizes), _address(types), len(grads), scale, kind,
                           norm.data_ptr(), wsp, ws.numel(), _stream(device)), "grad_norm")
    return norm


def clip_grads(grads, max_norm: float, scale: float = 1.0, norm_type: float = 2.0, out=None, stream=None):
    """Norm of scale * g over all tensors together; the gradients are scaled down to max_norm where it is above.

    out[i] = grads[i] * scale * min(1, max_norm / norm), in place without `out`.  grads, out: contiguous CUDA tensors, bf16
    or fp32 each, out[i] of grads[i]'s shape and of either type (fp32 is what adamw takes).  A NaN norm makes all values
    NaN."""
    grads, out = list(grads), None if out is None else list(out)
    if stream is not None:
        return _on(stream, clip_grads, grads, max_norm, scale=scale, norm_type=norm_type, out=out)
    kind = _norm_kind(norm_type)
    device = _device_of(grads)
    pointers, sizes, types = _tensors(grads, device, "grads")
    out_pointers, out_types = pointers, types
    if out is not None:
        if [t.shape for t in out] != [t.shape for t in grads]:
            raise ValueError("out must have a tensor of the same shape for each of grads")
        out_pointers, _, out_types = _tensors(out, device, "out")
    norm = torch.empty((), dtype=torch.float32, device=device)
    ws, wsp = _workspace(lib().grad_norm_workspace(len(grads)), device, "clip_grads")
    _check(lib().clip_grads(_address(pointers), _address(sizes), _address(types), _address(out_pointers),
                            _address(out_types), len(grads), scale, max_norm, kind, norm.data_ptr(), wsp, ws.numel(),
                            _stream(device)), "clip_grads")
    return norm
