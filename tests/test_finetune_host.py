"""Refusals of the fine-tuning operators (include/finetune.h): sizes, types,
pointers, alignment, numbers and workspaces are checked on the host before any
device work, and the binding refuses tensors it cannot pass (no GPU needed)."""
import ctypes
import math
from array import array

import pytest

import spectral_corrected_optimizer_gb300 as so
from spectral_corrected_optimizer_gb300 import build as sob
from spectral_corrected_optimizer_gb300 import finetune as ft

torch = pytest.importorskip("torch")
P = ctypes.c_void_p(1 << 20)
ODD = ctypes.c_void_p((1 << 20) + 1)
BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    sob.build()
    return so.lib()


def test_layernorm_refusals(lib):
    def fwd(x=P, r=P, g=P, b=P, t=0, eps=1e-5, s=P, y=P, mu=P, rs=P, rows=3, dim=16):
        return lib.layernorm_forward(x, r, g, b, t, eps, s, y, mu, rs, rows, dim, None)
    for bad in (dict(x=None), dict(g=None), dict(s=None), dict(y=None), dict(mu=None), dict(rs=None), dict(t=2), dict(eps=-1.0),
                dict(eps=NAN), dict(rows=-1), dict(rows=1 << 31), dict(dim=0), dict(dim=32769)):
        assert fwd(**bad) == so.ERR_INVALID_ARG, bad
        assert b"layernorm_forward" in lib.specoptim_last_error()
    for bad in (dict(x=ODD), dict(r=ODD), dict(b=ODD), dict(g=ODD), dict(y=ODD), dict(s=ODD), dict(mu=ODD), dict(rs=ODD)):
        assert fwd(**bad) == so.ERR_MISALIGNED, bad
    assert fwd(rows=0, x=None, y=None) == so.OK

    need = lib.layernorm_backward_workspace(3, 16)

    def bwd(dy=P, ds=P, s=P, mu=P, rs=P, g=P, t=0, dx=P, dg=P, db=P, rows=3, dim=16, ws=P, n=BIG):
        return lib.layernorm_backward(dy, ds, s, mu, rs, g, t, dx, dg, db, rows, dim, ws, n, None)
    assert need > 0 and lib.layernorm_backward_workspace(3, 0) == -1 and lib.layernorm_backward_workspace(-1, 8) == -1
    for bad in (dict(dy=None), dict(s=None), dict(mu=None), dict(rs=None), dict(g=None), dict(dx=None), dict(dg=None),
                dict(ws=None), dict(n=0), dict(t=9), dict(dim=-4)):
        assert bwd(**bad) == so.ERR_INVALID_ARG, bad
    for bad in (dict(dy=ODD), dict(ds=ODD), dict(s=ODD), dict(dx=ODD), dict(dg=ODD), dict(db=ODD), dict(ws=ODD), dict(mu=ODD)):
        assert bwd(**bad) == so.ERR_MISALIGNED, bad


def test_head_logp_refusals(lib):
    def fwd(h=P, w=P, t=P, ib=8, tokens=4, vocab=9, dim=8, logp=P, kept=P, ws=P, n=BIG):
        return lib.head_logp(h, w, t, ib, -100, tokens, vocab, dim, logp, kept, ws, n, None)
    need = lib.head_logp_workspace(4, 9, 8)
    for bad in (dict(h=None), dict(w=None), dict(t=None), dict(ib=3), dict(tokens=-1), dict(vocab=0), dict(dim=0), dict(logp=None),
                dict(kept=None), dict(ws=None), dict(n=need - 1), dict(dim=65537)):
        assert fwd(**bad) == so.ERR_INVALID_ARG, bad
    for bad in (dict(h=ODD), dict(w=ctypes.c_void_p((1 << 20) + 8)), dict(t=ODD), dict(logp=ODD), dict(kept=ODD), dict(ws=ODD)):
        assert fwd(**bad) == so.ERR_MISALIGNED, bad
    assert fwd(tokens=0, h=None, t=None, logp=None, kept=None) == so.OK

    need = lib.head_logp_backward_workspace(4, 9, 8)

    def bwd(d=P, kept=P, h=P, w=P, t=P, ib=8, tokens=4, vocab=9, dim=8, dh=P, dw=P, dt=1, ws=P, n=BIG):
        return lib.head_logp_backward(d, kept, h, w, t, ib, -100, tokens, vocab, dim, dh, dw, dt, 0, ws, n, None)
    for bad in (dict(d=None), dict(kept=None), dict(h=None), dict(w=None), dict(t=None), dict(ib=5), dict(vocab=0), dict(dh=None),
                dict(dw=None), dict(dt=2), dict(ws=None), dict(n=need - 1)):
        assert bwd(**bad) == so.ERR_INVALID_ARG, bad
    for bad in (dict(d=ODD), dict(kept=ODD), dict(dh=ODD), dict(dw=ODD), dict(t=ODD)):
        assert bwd(**bad) == so.ERR_MISALIGNED, bad
    # no statistics are formed: the workspace is smaller than that of the loss with its gradients
    assert lib.head_logp_backward_workspace(8192, 128256, 2048) < lib.head_loss_grad_workspace(8192, 128256, 2048)


def test_preference_refusals(lib):
    need = lib.preference_loss_workspace(100, 1 << 20)

    def call(x=P, r=P, m=P, o=P, ob=8, pairs=2, tokens=40, kind=0, beta=0.1, eps=0.0, scale=1.0, loss=P, pl=P, rw=P, d=P, ws=P, n=BIG):
        return lib.preference_loss(x, r, m, o, ob, pairs, tokens, kind, beta, eps, 0, 1, scale, loss, pl, rw, d, ws, n, None)
    # few sequences need no workspace
    assert need > 0 and lib.preference_loss_workspace(2, 40) == 0
    assert lib.preference_loss_workspace(-1, 4) == -1 and lib.preference_loss_workspace(1, -4) == -1
    for bad in (dict(x=None), dict(o=None), dict(loss=None), dict(pl=None), dict(rw=None), dict(d=None), dict(ob=2),
                dict(pairs=100, tokens=1 << 20, ws=None), dict(pairs=100, tokens=1 << 20, n=need - 1), dict(pairs=-1), dict(pairs=1 << 30), dict(tokens=-1), dict(kind=3), dict(kind=-1), dict(beta=0.0), dict(beta=-1.0),
                dict(beta=NAN), dict(beta=INF), dict(eps=-0.1), dict(eps=0.6), dict(eps=NAN), dict(eps=0.1, kind=1), dict(scale=INF),
                dict(scale=NAN)):
        assert call(**bad) == so.ERR_INVALID_ARG, bad
        assert b"preference_loss" in lib.specoptim_last_error()
    for bad in (dict(x=ODD), dict(r=ODD), dict(o=ODD), dict(loss=ODD), dict(pl=ODD), dict(rw=ODD), dict(d=ODD), dict(ws=ODD)):
        assert call(**bad) == so.ERR_MISALIGNED, bad


def test_policy_refusals(lib):
    def call(x=P, old=P, r=P, m=P, a=P, per=0, o=P, ob=8, count=2, tokens=40, low=0.2, high=0.2, kl=0.1, red=0, scale=1.0, loss=P,
             parts=P, d=P, ws=P, n=BIG):
        return lib.policy_loss(x, old, r, m, a, per, o, ob, count, tokens, low, high, kl, red, scale, loss, parts, d, ws, n, None)
    need = lib.policy_loss_workspace(100, 1 << 20)
    assert need > 0 and lib.policy_loss_workspace(2, 40) == 0 and lib.policy_loss_workspace(-1, 4) == -1
    for bad in (dict(x=None), dict(old=None), dict(a=None), dict(loss=None), dict(parts=None), dict(d=None), dict(ob=1),
                dict(count=100, tokens=1 << 20, ws=None), dict(count=100, tokens=1 << 20, n=need - 1),
                dict(count=-1), dict(tokens=-1), dict(low=-0.1), dict(low=1.1), dict(low=NAN), dict(high=-0.1), dict(high=NAN),
                dict(kl=NAN), dict(kl=INF), dict(r=None), dict(red=3), dict(scale=NAN), dict(o=None), dict(o=None, count=1, per=1)):
        assert call(**bad) == so.ERR_INVALID_ARG, bad
        assert b"policy_loss" in lib.specoptim_last_error()
    for bad in (dict(x=ODD), dict(old=ODD), dict(r=ODD), dict(a=ODD), dict(o=ODD), dict(loss=ODD), dict(parts=ODD), dict(d=ODD),
                dict(ws=ODD)):
        assert call(**bad) == so.ERR_MISALIGNED, bad


def host_array(kind, values):
    a = array(kind, values)
    return a, a.buffer_info()[0]


def test_clip_refusals(lib):
    where = 1 << 20

    def call(clip=True, at=(where, where + 4096), sizes=(100, 50), types=(1, 0), outs=(where, where + 4096), out_types=(1, 0), count=2,
             scale=1.0, most=1.0, kind=0, norm=P, ws=P, n=BIG, null=()):
        hold = [host_array("Q", at), host_array("q", sizes), host_array("i", types), host_array("Q", outs), host_array("i", out_types)]
        p = [None if i in null else h[1] for i, h in enumerate(hold)]
        if clip:
            return lib.clip_grads(*p, count, scale, most, kind, norm, ws, n, None)
        return lib.grad_norm(*p[:3], count, scale, kind, norm, ws, n, None)
    assert lib.grad_norm_workspace(0) > 0 and lib.grad_norm_workspace(-1) == -1
    assert lib.grad_norm_workspace(5000) > lib.grad_norm_workspace(5)
    for clip in (True, False):
        for bad in (dict(count=-1), dict(kind=2), dict(scale=INF), dict(scale=NAN), dict(norm=None), dict(ws=None), dict(types=(1, 2)),
                    dict(sizes=(-1, 5)), dict(at=(0, where)), dict(null=(0,)), dict(null=(1,)), dict(null=(2,))):
            assert call(clip=clip, **bad) == so.ERR_INVALID_ARG, bad
        for bad in (dict(at=(where + 1, where)), dict(norm=ODD), dict(ws=ODD)):
            assert call(clip=clip, **bad) == so.ERR_MISALIGNED, bad
    for bad in (dict(most=-1.0), dict(most=NAN), dict(null=(3,)), dict(null=(4,)), dict(out_types=(1, 5)), dict(outs=(where, 0)),
                dict(outs=(where, where + 399)), dict(outs=(where + 200, where + 8192)), dict(outs=(where + 4096, where)),
                dict(out_types=(0, 0)), dict(at=(where, where)), dict(outs=(where + 8192, where + 8192))):
        assert call(**bad) == (so.ERR_MISALIGNED if bad.get("outs") == (where, where + 399) else so.ERR_INVALID_ARG), bad
    assert call(outs=(where, where + 4097)) == so.ERR_MISALIGNED
    # tensors without values are not looked at
    assert call(sizes=(0, -5)) == so.ERR_INVALID_ARG
    assert call(sizes=(0, 0), at=(0, 1), outs=(0, 3), n=0) == so.ERR_INVALID_ARG and b"workspace" in lib.specoptim_last_error()


def test_binding_refuses_tensors_it_cannot_pass():
    bf = torch.bfloat16
    t, ids, f = torch.zeros(9, 8, dtype=bf), torch.zeros(9, dtype=torch.int64), torch.zeros(9)
    off = torch.tensor([0, 4, 9])
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        ft.layer_norm(t.half(), None, t[0].half())
    with pytest.raises(ValueError, match="CUDA"):
        ft.layer_norm(t, t, t[0], t[0])
    with pytest.raises(ValueError, match="bfloat16"):
        ft.head_logp(t.float(), t, ids)
    with pytest.raises(ValueError, match="accumulate"):
        ft.head_logp_backward(f, torch.zeros(3, 9), t, t, ids, accumulate=True)
    with pytest.raises(ValueError, match="kind"):
        ft.preference_loss(f, f, off, kind="other")
    with pytest.raises(ValueError, match="reduction"):
        ft.preference_loss(f, f, off, reduction="none")
    with pytest.raises(ValueError, match="logp must be torch.float32"):
        ft.preference_loss(f.double(), f, off)
    with pytest.raises(ValueError, match="CUDA"):
        ft.preference_loss(f, f, off)
    with pytest.raises(ValueError, match="reduction"):
        ft.policy_loss(f, f, f, reduction="mean")
    with pytest.raises(ValueError, match="CUDA"):
        ft.policy_loss(f, f, f)
    with pytest.raises(ValueError, match="norm_type"):
        ft.grad_norm([f], norm_type=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        ft.grad_norm([f])
    with pytest.raises(ValueError, match="CUDA"):
        ft.clip_grads([f], 1.0)
    assert ft._norm_kind(2) == 0 and ft._norm_kind(math.inf) == 1


class Fake:
    """Stands in for a CUDA tensor where only its description is asked for."""

    def __init__(self, shape, dtype=torch.float32, contiguous=True):
        self.t = torch.empty(shape, dtype=dtype, device="meta")
        self.dtype, self.shape, self.device, self.is_cuda, self.contiguous = dtype, self.t.shape, torch.device("cuda", 0), True, contiguous

    def numel(self):
        return self.t.numel()

    def dim(self):
        return self.t.dim()

    def is_contiguous(self):
        return self.contiguous

    def data_ptr(self):
        return 1 << 20


def test_binding_refuses_shapes_and_ambiguous_calls():
    f, off = Fake(9), Fake(3, torch.int64)
    with pytest.raises(ValueError, match="ref_logp must be"):
        ft.preference_loss(f, Fake(8), off)
    with pytest.raises(ValueError, match="mask must be"):
        ft.preference_loss(f, f, off, mask=Fake(9))
    with pytest.raises(ValueError, match="mask must be"):
        ft.preference_loss(f, f, off, mask=Fake(8, torch.bool))
    with pytest.raises(ValueError, match="offsets must be int32"):
        ft.preference_loss(f, f, Fake(3))
    with pytest.raises(ValueError, match="offsets must be int32"):
        ft.preference_loss(f, f, Fake(0, torch.int64))
    with pytest.raises(ValueError, match="pairs"):
        ft.preference_loss(f, f, Fake(4, torch.int64))
    with pytest.raises(ValueError, match="contiguous"):
        ft.preference_loss(Fake(9, contiguous=False), f, off)
    with pytest.raises(ValueError, match="kl_coef needs"):
        ft.policy_loss(f, f, f, kl_coef=0.1)
    with pytest.raises(ValueError, match="old_logp"):
        ft.policy_loss(f, None, f)
    with pytest.raises(ValueError, match="without offsets"):
        ft.policy_loss(f, f, Fake(2))
    with pytest.raises(ValueError, match="advantages must be"):
        ft.policy_loss(f, f, Fake(3), off)
    with pytest.raises(ValueError, match="per_sequence"):
        ft.policy_loss(f, f, f, Fake(10, torch.int64))
    with pytest.raises(ValueError, match="same shape"):
        ft.clip_grads([f], 1.0, out=[Fake(8)])
    with pytest.raises(ValueError, match="contiguous"):
        ft.grad_norm([f, Fake(9, contiguous=False)])
