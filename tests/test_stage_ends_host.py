"""Refusals of the stage-end operators (include/stage_ends.h): sizes, types,
pointers, alignment and workspaces are checked on the host before any device
work, and the binding refuses tensors it cannot pass (no GPU needed)."""
import ctypes

import pytest

import spectral_corrected_optimizer_gb300 as so
from spectral_corrected_optimizer_gb300 import build as sob
from spectral_corrected_optimizer_gb300 import stage_ends as se

torch = pytest.importorskip("torch")
P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    sob.build()
    return so.lib()


def test_embed_lookup_refusals(lib):
    def call(table=P, tt=0, ids=P, ib=8, tokens=4, vocab=9, dim=8, out=P, ot=0):
        return lib.embed_lookup(table, tt, ids, ib, tokens, vocab, dim, 1.0, out, ot, None)
    for bad in (dict(tt=2), dict(ot=-1), dict(ib=2), dict(tokens=-1), dict(vocab=0), dict(dim=0), dict(table=None),
                dict(ids=None), dict(out=None), dict(tokens=1 << 31), dict(vocab=1 << 31), dict(dim=1 << 21)):
        assert call(**bad) == so.ERR_INVALID_ARG, bad
        assert b"embed_lookup" in lib.specoptim_last_error()
    for bad in (dict(table=ODD), dict(ids=ODD), dict(out=ODD)):
        assert call(**bad) == so.ERR_MISALIGNED, bad
    assert call(tokens=0, table=None, ids=None, out=None) == so.OK


def test_embed_grad_refusals(lib):
    def call(ids=P, ib=8, dy=P, dt=0, tokens=4, vocab=9, dim=8, pad=-1, grad=P, gt=1, ws=P, n=BIG):
        return lib.embed_grad(ids, ib, dy, dt, tokens, vocab, dim, pad, 1.0, grad, gt, 0, ws, n, None)
    need = lib.embed_grad_workspace(4, 9, 8)
    assert need > 0 and lib.embed_grad_workspace(-1, 9, 8) == -1 and lib.embed_grad_workspace(4, 0, 8) == -1
    for bad in (dict(ib=1), dict(dt=5), dict(gt=5), dict(pad=9), dict(pad=-2), dict(grad=None), dict(dy=None),
                dict(ids=None), dict(ws=None), dict(n=need - 1), dict(dim=0)):
        assert call(**bad) == so.ERR_INVALID_ARG, bad
    for bad in (dict(dy=ODD), dict(grad=ODD), dict(ids=ODD), dict(ws=ODD)):
        assert call(**bad) == so.ERR_MISALIGNED, bad


def test_resnorm_refusals(lib):
    def fwd(x=P, r=P, g=P, t=0, eps=1e-5, s=P, y=P, q=P, sc=P, rs=P, rows=3, dim=16):
        return lib.resnorm_forward(x, r, g, t, eps, s, y, q, sc, rs, rows, dim, None)
    for bad in (dict(x=None), dict(g=None), dict(s=None), dict(y=None), dict(q=None), dict(sc=None), dict(rs=None),
                dict(t=3), dict(eps=-1.0), dict(eps=float("nan")), dict(rows=-1), dict(dim=0), dict(dim=32769)):
        assert fwd(**bad) == so.ERR_INVALID_ARG, bad
    for bad in (dict(x=ODD), dict(r=ODD), dict(y=ODD), dict(sc=ODD), dict(rs=ODD)):
        assert fwd(**bad) == so.ERR_MISALIGNED, bad
    assert fwd(rows=0, x=None, y=None) == so.OK

    def bwd(dy=P, ds=P, q=P, sc=P, rs=P, g=P, t=0, dx=P, dg=P, y=P, rows=3, dim=16, ws=P, n=BIG):
        return lib.resnorm_backward(dy, ds, q, sc, rs, g, t, dx, dg, y, rows, dim, ws, n, None)
    assert lib.resnorm_backward_workspace(3, 0) == -1
    for bad in (dict(dy=None), dict(q=None), dict(sc=None), dict(rs=None), dict(g=None), dict(dx=None), dict(dg=None),
                dict(ws=None), dict(n=0), dict(t=9), dict(dim=-4)):
        assert bwd(**bad) == so.ERR_INVALID_ARG, bad
    for bad in (dict(dy=ODD), dict(ds=ODD), dict(dx=ODD), dict(dg=ODD), dict(y=ODD), dict(ws=ODD)):
        assert bwd(**bad) == so.ERR_MISALIGNED, bad
    assert lib.resnorm_recompute(None, P, P, P, 0, P, 3, 16, None) == so.ERR_INVALID_ARG
    assert lib.resnorm_recompute(P, P, P, ODD, 0, P, 3, 16, None) == so.ERR_MISALIGNED


def test_head_refusals(lib):
    def loss(h=P, w=P, t=P, ib=8, tokens=4, vocab=9, dim=8, out=P, rows=P, ws=P, n=BIG):
        return lib.head_loss(h, w, t, ib, -100, tokens, vocab, dim, 1, out, rows, ws, n, None)
    need = lib.head_loss_workspace(4, 9, 8)
    for bad in (dict(h=None), dict(w=None), dict(t=None), dict(ib=3), dict(tokens=-1), dict(vocab=0), dict(dim=0),
                dict(out=None), dict(rows=None), dict(ws=None), dict(n=need - 1), dict(dim=65537),
                dict(tokens=(1 << 24) + 1)):
        assert loss(**bad) == so.ERR_INVALID_ARG, bad
    for bad in (dict(h=ODD), dict(w=ctypes.c_void_p((1 << 20) + 8)), dict(t=ODD), dict(out=ODD), dict(rows=ODD),
                dict(ws=ODD)):
        assert loss(**bad) == so.ERR_MISALIGNED, bad

    def grad(dh=P, dw=P, dt=1, n=BIG, h=P):
        return lib.head_loss_grad(h, P, P, 8, -100, 4, 9, 8, 1, 1.0, P, P, dh, dw, dt, 0, P, n, None)
    for bad in (dict(dh=None), dict(dw=None), dict(dt=2), dict(n=lib.head_loss_grad_workspace(4, 9, 8) - 1), dict(h=None)):
        assert grad(**bad) == so.ERR_INVALID_ARG, bad
    for bad in (dict(dh=ODD), dict(dw=ODD)):
        assert grad(**bad) == so.ERR_MISALIGNED, bad
    assert lib.head_loss_workspace(4, -1, 8) == -1 and lib.head_loss_grad_workspace(-1, 9, 8) == -1


def test_workspaces_grow_with_the_tokens_not_with_the_logits(lib):
    # the whole point of working in pieces: far below tokens x vocabulary
    tokens, vocab, dim = 65536, 128256, 2048
    logits = tokens * vocab * 2
    assert lib.head_loss_workspace(tokens, vocab, dim) < logits / 16
    assert lib.head_loss_grad_workspace(tokens, vocab, dim) < logits / 6


def test_binding_refuses_tensors_it_cannot_pass():
    bf = torch.bfloat16
    t, ids = torch.zeros(9, 8, dtype=bf), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        se.embed_lookup(t, ids)
    with pytest.raises(ValueError, match="int32 or int64"):
        se.embed_lookup(t, ids.float())
    with pytest.raises(ValueError, match="dtype"):
        se.embed_lookup(t, ids, dtype=torch.float16)
    with pytest.raises(ValueError, match="accumulate"):
        se.embed_grad(ids, t[:4], 9, accumulate=True)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        se.residual_norm(t.half(), None, t[0].half())
    with pytest.raises(ValueError, match="CUDA"):
        se.residual_norm(t, t, t[0])
    with pytest.raises(ValueError, match="reduction"):
        se.head_loss(t, t, ids, reduction="none")
    with pytest.raises(ValueError, match="bfloat16"):
        se.head_loss(t.float(), t, ids)
