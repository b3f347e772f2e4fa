"""GPU parity of the stage-end operators (include/stage_ends.h) with their
definitions in float64.

u16 = 2^-8 is the unit roundoff of bf16, u32 = 2^-24 that of fp32.
- lookup: one fp32 product, one rounding: bit-exact.
- embedding gradient: a row of n tokens is a sum of n fp32 values in some order,
  one product with the scale: |error| <= (n + 1) u32 sum |dy| |scale|, and u16 of
  the result where it is stored in bf16.
- norm: s, the 8-bit values and their scales follow fp32 operations one by one:
  bit-exact.  rstd sums squares over at most 64 values in a row, 5 shuffle steps
  and 16 warps: relative error below 100 u32, and so y before its rounding.
  Backward: the mean is such a sum too: 100 u32 of the magnitudes of dx's terms;
  dgamma adds at most `rows` terms: (rows + 10) u32 of their magnitudes.
- head: a logit is the exact bf16 products added 16 at a time into fp32, whose
  adder may truncate: (dim / 16 + 4) 2^-23 of sum |h||w| =: e, twice in a row's
  loss, plus 2^-22 (|lse| + 8) for exp and log.  The gradients' probabilities are
  off by e relatively and are rounded to bf16: (u16 + e) of sum |d||W| (or
  sum |d||h|) beside the rounding of the result.
"""
import math

import pytest
import torch

import stage_ends_ref as ref
from gpu_util import Guarded, ensure_lib

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.fixture(autouse=True)
def _clean_flag(_lib):
    yield
    import spectral_corrected_optimizer_gb300 as so
    so.check_device()


def se():
    from spectral_corrected_optimizer_gb300 import stage_ends
    return stage_ends


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, shape, dtype=FP, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(dtype)


def u_of(dtype):
    return U16 if dtype == BF else U32


# ---------------------------------------------------------------- embedding

LOOKUPS = [(1, 7, 1), (3, 50, 8), (37, 333, 100), (5, 1000, 4096), (2500, 97, 257), (5000, 1201, 64), (0, 5, 16)]


@pytest.mark.parametrize("tokens,vocab,dim", LOOKUPS)
@pytest.mark.parametrize("tin,tout", [(BF, BF), (FP, BF), (FP, FP), (BF, FP)])
@pytest.mark.parametrize("idt", [torch.int64, torch.int32])
def test_lookup_bit_exact(tokens, vocab, dim, tin, tout, idt):
    g = gen(tokens + dim)
    table, scale = randn(g, (vocab, dim), tin), math.sqrt(dim)
    ids = torch.randint(0, vocab, (tokens,), generator=g, dtype=idt)
    out = Guarded((tokens, dim), tout)
    got = se().embed_lookup(table.cuda(), ids.cuda(), scale=scale, out=out.t)
    want = (table[ids.long()].float() * torch.tensor(scale, dtype=FP)).to(tout)
    assert torch.equal(got.cpu(), want) and out.intact()


def test_lookup_of_unaligned_views_and_other_shapes():
    g = gen(3)
    flat = randn(g, (41 * 24 + 1,), BF).cuda()
    table = flat[1:].view(41, 24)  # 2-byte aligned only
    ids = torch.randint(0, 41, (2, 3, 5), generator=g).cuda()
    got = se().embed_lookup(table, ids)
    assert got.shape == (2, 3, 5, 24) and torch.equal(got, table[ids])


GRADS = [(1, 5, 8), (2, 3, 1), (9, 40, 24), (64, 7, 100), (777, 501, 264), (3000, 100000, 40), (2100, 600, 2056),
         (70000, 1000, 16), (5000, 2, 48)]


def zipf(g, tokens, vocab):
    u = torch.rand(tokens, generator=g, dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)


def check_grad(got, ids, dy, vocab, scale, padding=None, before=None):
    want, mag, n = ref.embed_grad(ids, dy, vocab, scale, padding)
    tol = (n[:, None] + 1) * U32 * mag
    if before is not None:
        want = want + before.double()
        tol = tol + U32 * (mag + before.double().abs())
    tol = tol + (U16 * want.abs() if got.dtype == BF else U32 * want.abs())
    err = (got.cpu().double() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


@pytest.mark.parametrize("tokens,vocab,dim", GRADS)
@pytest.mark.parametrize("din,dout", [(BF, FP), (BF, BF), (FP, FP)])
def test_embed_grad(tokens, vocab, dim, din, dout):
    g = gen(tokens * 3 + dim)
    ids, dy = zipf(g, tokens, vocab), randn(g, (tokens, dim), din)
    out = Guarded((vocab, dim), dout, fill=7.0)
    got = se().embed_grad(ids.cuda(), dy.cuda(), vocab, scale=1.5, out=out.t)
    check_grad(got, ids, dy, vocab, 1.5)
    assert out.intact()
    absent = torch.bincount(ids, minlength=vocab) == 0
    assert bool((got.cpu()[absent] == 0).all())
    # the same bits every time: no sum depends on timing
    assert torch.equal(got, se().embed_grad(ids.cuda(), dy.cuda(), vocab, scale=1.5, dtype=dout))


@pytest.mark.parametrize("dout", [FP, BF])
@pytest.mark.parametrize("dim", [40, 13])
def test_embed_grad_adds_to_a_gradient_and_leaves_other_rows(dim, dout):
    g = gen(5)
    ids, dy = zipf(g, 400, 90).to(torch.int32), randn(g, (400, dim), BF)
    before = randn(g, (90, dim), dout)
    got = se().embed_grad(ids.cuda(), dy.cuda(), 90, out=before.cuda(), accumulate=True)
    check_grad(got, ids, dy, 90, 1.0, before=before)
    absent = torch.bincount(ids.long(), minlength=90) == 0
    assert bool(absent.any()) and torch.equal(got.cpu()[absent], before[absent])


@pytest.mark.parametrize("dim", [8, 248, 256, 1024, 2040, 2048, 4096])
@pytest.mark.parametrize("tokens", [700, 2600, 8192, 20000])
def test_embed_grad_workspace_serves_every_alignment(tokens, dim):
    # the chunks, and with them the partial sums, differ between aligned and unaligned rows
    g = gen(tokens + dim)
    ids, dy = zipf(g, tokens, 40), randn(g, (tokens, dim), BF)
    for given in (dy.cuda(), shifted(dy, 3)):
        check_grad(se().embed_grad(ids.cuda(), given, 40), ids, dy, 40, 1.0)


@pytest.mark.parametrize("ids", [[4] * 700, list(range(600)), [0, 599] * 300, [599] * 3 + [0] * 200 + [300] * 500])
def test_embed_grad_of_extreme_orders(ids):
    ids = torch.tensor(ids)
    dy = randn(gen(8), (len(ids), 72), BF)
    check_grad(se().embed_grad(ids.cuda(), dy.cuda(), 600), ids, dy, 600, 1.0)


def test_embed_grad_padding_and_no_tokens():
    g = gen(9)
    ids, dy = zipf(g, 300, 20), randn(g, (300, 32), BF)
    got = se().embed_grad(ids.cuda(), dy.cuda(), 20, padding_idx=0)
    check_grad(got, ids, dy, 20, 1.0, padding=0)
    assert bool((got[0] == 0).all())
    none = se().embed_grad(ids[:0].cuda(), dy[:0].cuda(), 20)
    assert none.shape == (20, 32) and bool((none == 0).all())


def test_ids_outside_the_vocabulary_are_skipped_and_reported():
    import spectral_corrected_optimizer_gb300 as so
    g = gen(10)
    table, dy = randn(g, (30, 16), BF).cuda(), randn(g, (6, 16), BF)
    ids = torch.tensor([3, 30, -1, 29, 2 ** 40, 3])
    got = se().embed_lookup(table, ids.cuda())
    with pytest.raises(so.SpecOptimError, match="token id") as e:
        so.check_device()
    assert e.value.code == so.ERR_BOUNDS
    assert bool((got[[1, 2, 4]] == 0).all()) and torch.equal(got[[0, 3, 5]], table[[3, 29, 3]])
    check_grad(se().embed_grad(ids.cuda(), dy.cuda(), 30), ids, dy, 30, 1.0)
    with pytest.raises(so.SpecOptimError, match="token id"):
        so.check_device()


def test_embed_grad_is_the_lookups_adjoint():
    # <lookup(E), dy> = <E, grad(dy)>: the lookup is linear, so this is its difference quotient
    g = gen(11)
    ids, dy, table = zipf(g, 500, 60), randn(g, (500, 40)), randn(g, (60, 40))
    y = se().embed_lookup(table.cuda(), ids.cuda(), scale=0.7)
    d = se().embed_grad(ids.cuda(), dy.cuda(), 60, scale=0.7)
    a, b = (y.cpu().double() * dy).sum(), (d.cpu().double() * table).sum()
    mag = (y.cpu().double() * dy).abs().sum()
    assert abs(a - b) <= 502 * U32 * mag


# ---------------------------------------------------------------- residual norm

NORMS = [(1, 1), (3, 7), (5, 128), (4, 129), (17, 256), (9, 1001), (6, 2048), (3, 4096), (2, 8200), (2, 12345),
         (1, 32768), (700, 264)]


def norm_inputs(rows, dim, dtype, residual, seed=0):
    g = gen(seed + rows * 7 + dim)
    x = torch.randn(rows, dim, generator=g) * torch.exp(torch.randn(rows, 1, generator=g))
    x[:, ::97] *= 30
    r = randn(g, (rows, dim), dtype) if residual else None
    return x.to(dtype), r, (1 + 0.3 * torch.randn(dim, generator=g)).to(dtype), g


@pytest.mark.parametrize("rows,dim", NORMS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("residual", [True, False])
def test_residual_norm_and_its_backward(rows, dim, dtype, residual):
    x, r, gamma, g = norm_inputs(rows, dim, dtype, residual)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    kept, s, y = se().residual_norm(x.cuda(), cuda(r), gamma.cuda(), 1e-5)
    want_s = x if r is None else (x.float() + r.float()).to(dtype)
    assert torch.equal(s.cpu(), want_s)
    q, scale = ref.checkpoint32(want_s)
    assert torch.equal(kept.scale.cpu(), scale)
    assert torch.equal(kept.q.cpu().view(torch.uint8), q.view(torch.uint8))
    want_y, rstd = ref.norm_forward(want_s, gamma, 1e-5)
    assert bool(((kept.rstd.cpu().double() - rstd).abs() <= 100 * U32 * rstd).all())
    assert bool(((y.cpu().double() - want_y).abs() <= (u_of(dtype) + 104 * U32) * want_y.abs()).all())

    dy = randn(g, (rows, dim), dtype)
    ds = randn(g, (rows, dim), dtype, 0.3) if residual else None
    dx, dgamma, y2 = se().residual_norm_backward(dy.cuda(), kept, gamma.cuda(), ds=cuda(ds), recompute=True)
    w_dx, m_dx, w_dg, m_dg, w_y = ref.norm_backward(dy, ds, kept.q.cpu(), kept.scale.cpu(), kept.rstd.cpu(), gamma)
    assert bool(((dx.cpu().double() - w_dx).abs() <= u_of(dtype) * w_dx.abs() + 100 * U32 * m_dx).all())
    assert bool(((dgamma.cpu().double() - w_dg).abs() <= (rows + 10) * U32 * m_dg).all())
    assert bool(((y2.cpu().double() - w_y).abs() <= (u_of(dtype) + 4 * U32) * w_y.abs()).all())
    assert torch.equal(se().residual_norm_recompute(kept, gamma.cuda()), y2)
    again = se().residual_norm_backward(dy.cuda(), kept, gamma.cuda(), ds=cuda(ds))
    assert again[2] is None and torch.equal(again[0], dx) and torch.equal(again[1], dgamma)


def test_residual_norm_many_rows():
    # more rows than blocks: every block walks over several rows
    x, r, gamma, g = norm_inputs(20000, 72, BF, True)
    kept, s, y = se().residual_norm(x.cuda(), r.cuda(), gamma.cuda(), 1e-6)
    want_s = (x.float() + r.float()).to(BF)
    q, scale = ref.checkpoint32(want_s)
    assert torch.equal(s.cpu(), want_s) and torch.equal(kept.q.cpu().view(torch.uint8), q.view(torch.uint8))
    want_y, _ = ref.norm_forward(want_s, gamma, 1e-6)
    assert bool(((y.cpu().double() - want_y).abs() <= (U16 + 104 * U32) * want_y.abs()).all())
    dy = randn(g, x.shape, BF)
    dx, dgamma, _ = se().residual_norm_backward(dy.cuda(), kept, gamma.cuda())
    w = ref.norm_backward(dy, None, kept.q.cpu(), kept.scale.cpu(), kept.rstd.cpu(), gamma)
    assert bool(((dx.cpu().double() - w[0]).abs() <= U16 * w[0].abs() + 100 * U32 * w[1]).all())
    assert bool(((dgamma.cpu().double() - w[2]).abs() <= 20010 * U32 * w[3]).all())


def test_residual_norm_zero_tiny_and_non_finite_rows():
    x = torch.zeros(7, 300)
    x[1] = 1e-38                      # below the smallest scale's 448th
    x[2, 5] = float("inf")            # its group is lost, the other groups are kept
    x[3, 299] = float("nan")
    x[4] = torch.linspace(-3e38, 3e38, 300)  # its fp32 step overflows: infinities and NaN throughout
    x[5] = 1.0
    x[6] = torch.arange(-150, 150) * 2e36
    gamma = torch.ones(300)
    kept, s, y = se().residual_norm(x.cuda(), None, gamma.cuda(), 1e-5)
    back = ref.dequantise(kept.q.cpu(), kept.scale.cpu())
    assert bool((back[0] == 0).all()) and bool((y[0] == 0).all())
    assert bool(((back[1] - 1e-38).abs() <= 2.0 ** -126 * 2.0 ** -4).all())
    assert bool(back[2, :128].isnan().all()) and bool((back[2, 128:] == 0).all())
    assert bool(back[3, 256:].isnan().all()) and bool((back[3, :256] == 0).all())
    assert bool(x[4].isfinite().all()) or bool(back[4].isnan().any())
    assert bool((back[6] - x[6].double()).abs().max() <= 3e38 * 2.0 ** -4)
    q, scale = ref.checkpoint32(x)
    assert torch.equal(scale, kept.scale.cpu())
    assert torch.equal(back.nan_to_num(nan=-1.0), ref.dequantise(q, scale).nan_to_num(nan=-1.0))
    assert torch.equal(back[5].view(1, 300), ref.dequantise(torch.full((1, 300), 448.0), kept.scale.cpu()[5:6]))
    assert bool(((back[5] - 1).abs() <= U32).all())
    assert bool(y[2].isnan().any()) and bool(y[3].isnan().all())
    dx, dgamma, _ = se().residual_norm_backward(torch.ones(7, 300).cuda(), kept, gamma.cuda())
    assert bool(dx[[0, 1, 5]].isfinite().all())


def test_residual_norm_of_no_rows():
    gamma = torch.ones(64, dtype=BF).cuda()
    x = torch.empty(0, 64, dtype=BF).cuda()
    kept, s, y = se().residual_norm(x, x, gamma)
    dx, dgamma, _ = se().residual_norm_backward(x, kept, gamma)
    assert y.shape == (0, 64) and dx.shape == (0, 64) and bool((dgamma == 0).all())


def test_residual_norm_backward_against_differences():
    # values that 8 bits hold exactly: the checkpoint is the input, so the backward
    # pass has to match difference quotients of the forward pass itself
    g = gen(21)
    rows, dim, eps, step = 4, 256, 1e-3, 2.0 ** -7
    x = torch.randint(-8, 9, (rows, dim), generator=g).float() * 8
    x[:, 0] = x[:, 128] = 448.0
    gamma = 1 + 0.3 * torch.randn(dim, generator=g)
    dy, u = torch.randn(rows, dim, generator=g), torch.randn(rows, dim, generator=g)
    kept, _, _ = se().residual_norm(x.cuda(), None, gamma.cuda(), eps)
    assert torch.equal(ref.dequantise(kept.q.cpu(), kept.scale.cpu()), x.double())
    dx, dgamma, _ = se().residual_norm_backward(dy.cuda(), kept, gamma.cuda())
    f = lambda v: (ref.norm_forward(v, gamma, eps)[0] * dy.double()).sum(-1)  # noqa: E731
    diff = (f(x.double() + step * u) - f(x.double() - step * u)) / (2 * step)
    got = (dx.cpu().double() * u).sum(-1)
    # second-order term: (step / |x|)^2 of the quotient's magnitude, |x| ~ 50; fp32 sums of 256 terms
    mag = (dx.cpu().double() * u).abs().sum(-1)
    assert bool(((got - diff).abs() <= 1e-5 * mag).all())
    fg = (ref.norm_forward(x, torch.ones(dim), eps)[0] * dy.double()).sum(0)
    assert bool(((dgamma.cpu().double() - fg).abs() <= 1e-5 * (fg.abs() + 1)).all())


def shifted(t, by):
    """The same values in a contiguous CUDA view that begins `by` elements behind a 16-byte boundary."""
    buf = torch.empty(t.numel() + by, dtype=t.dtype, device="cuda")
    view = buf[by:].view(t.shape)
    view.copy_(t)
    return view


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim,by", [(256, 1), (131, 3), (9, 5)])
def test_operators_on_unaligned_views(dtype, dim, by):
    # tensors of one call that begin at different places between two 16-byte boundaries
    x, r, gamma, g = norm_inputs(30, dim, dtype, True, seed=5)
    kept, s, y = se().residual_norm(shifted(x, by), shifted(r, 2), shifted(gamma, 1), 1e-5)
    plain = se().residual_norm(x.cuda(), r.cuda(), gamma.cuda(), 1e-5)
    assert torch.equal(s, plain[1]) and torch.equal(kept.q.view(torch.uint8), plain[0].q.view(torch.uint8))
    want_y, _ = ref.norm_forward(s.cpu(), gamma, 1e-5)
    assert bool(((y.cpu().double() - want_y).abs() <= (u_of(dtype) + 104 * U32) * want_y.abs()).all())
    dy = randn(g, x.shape, dtype)
    kept = se().NormCheckpoint(shifted(kept.q.view(torch.uint8), by).view(torch.float8_e4m3fn), kept.scale, kept.rstd)
    dx, dgamma, y2 = se().residual_norm_backward(shifted(dy, 4), kept, shifted(gamma, 3), ds=shifted(r, by), recompute=True)
    w = ref.norm_backward(dy, r, kept.q.cpu(), kept.scale.cpu(), kept.rstd.cpu(), gamma)
    assert bool(((dx.cpu().double() - w[0]).abs() <= u_of(dtype) * w[0].abs() + 100 * U32 * w[1]).all())
    assert bool(((dgamma.cpu().double() - w[2]).abs() <= 40 * U32 * w[3]).all())
    assert bool(((y2.cpu().double() - w[4]).abs() <= (u_of(dtype) + 4 * U32) * w[4].abs()).all())
    assert torch.equal(se().residual_norm_recompute(kept, shifted(gamma, 5)), y2)

    ids = zipf(g, 30, 17)
    out = shifted(torch.zeros(17, dim, dtype=dtype), by)
    check_grad(se().embed_grad(shifted(ids, 1), shifted(dy, 3), 17, out=out), ids, dy, 17, 1.0)
    check_grad(se().embed_grad(ids.cuda(), shifted(dy, 6), 17, out=out, accumulate=True), ids, dy, 17, 1.0,
               before=ref.embed_grad(ids, dy, 17, 1.0)[0].to(dtype))
    table = randn(g, (17, dim), dtype)
    out = shifted(torch.zeros(30, dim, dtype=BF), 7)
    got = se().embed_lookup(shifted(table, by), ids.cuda(), scale=3.0, out=out)
    assert torch.equal(got.cpu(), (table[ids].float() * 3).to(BF))


@pytest.mark.parametrize("dim", [64, 72, 33])
def test_head_with_unaligned_hidden_states_and_gradient(dim):
    h, w, target = head_inputs(90, 700, dim, seed=9)
    dw = shifted(torch.zeros(700, dim), 1)
    loss, row_loss, dh, dw = se().head_loss_grad(shifted(h, 3), w.cuda(), shifted(target, 1), dw=dw)
    want = ref.head(h, w, target)
    check_loss(loss, row_loss, want, dim)
    check_grads(dh, dw, want, h, w)


# ---------------------------------------------------------------- head

HEADS = [(1, 3, 8), (1, 1000, 64), (5, 257, 72), (130, 300, 64), (128, 256, 128), (300, 1111, 200), (257, 5000, 136),
         (64, 40000, 64), (33, 900, 1001), (40, 513, 7), (700, 6000, 320)]


def head_inputs(tokens, vocab, dim, seed=0, ignored=0.0):
    g = gen(seed + tokens + vocab * 3 + dim * 7)
    w = randn(g, (vocab, dim), BF, 0.1)
    target = torch.randint(0, vocab, (tokens,), generator=g)
    h = (torch.randn(tokens, dim, generator=g) + 8 * torch.rand(tokens, 1, generator=g) * w[target].float()).to(BF)
    if ignored:
        target[torch.rand(tokens, generator=g) < ignored] = -100
    return h, w, target


def logit_error(want, dim):
    return (dim / 16 + 4) * 2.0 ** -23 * want["logit_mag"]


def check_loss(loss, row_loss, want, dim):
    tol = 2 * logit_error(want, dim) + 2.0 ** -22 * (want["lse"].abs() + 8)
    err = (row_loss.cpu().double() - want["row_loss"]).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    assert bool((row_loss.cpu()[~want["valid"]] == 0).all())
    f = want["loss_factor"]
    total = f * (tol * want["valid"]).sum() + 2.0 ** -20 * f * want["row_loss"].abs().sum()
    assert abs(float(loss) - float(want["loss"])) <= float(total)


def check_grads(dh, dw, want, h, w, before=None):
    d, e = want["d"].abs(), U16 + logit_error(want, h.shape[1])[:, None]
    g = abs(want["factor"])
    tol_h = g * e * (d @ w.double().abs())
    tol_w = g * ((d * e).T @ h.double().abs())
    want_h, want_w = want["dh"], want["dw"]
    if before is not None:
        want_w = want_w + before.double()
        tol_w = tol_w + U32 * before.double().abs()
    for got, full, tol in ((dh, want_h, tol_h), (dw, want_w, tol_w)):
        err = (got.cpu().double() - full).abs()
        tol = tol + (U16 if got.dtype == BF else U32) * full.abs() + 1e-30
        assert bool((err <= tol).all()), float((err / tol).max())
    # roundings are independent of each other: in norm they stay within one unit roundoff of bf16
    for got, full in ((dh, want_h), (dw, want_w)):
        norm = full.norm()
        if norm > 2.0 ** -126:  # below that neither type holds the values
            assert float((got.cpu().double() - full).norm() / norm) <= U16
    assert bool((dh.cpu()[~want["valid"]] == 0).all())


@pytest.mark.parametrize("tokens,vocab,dim", HEADS)
def test_head_loss(tokens, vocab, dim):
    h, w, target = head_inputs(tokens, vocab, dim)
    loss, row_loss = se().head_loss(h.cuda(), w.cuda(), target.cuda())
    check_loss(loss, row_loss, ref.head(h, w, target), dim)


@pytest.mark.parametrize("tokens", [1, 2, 4])
@pytest.mark.parametrize("vocab,dim", [(1, 8), (2, 5), (33, 64), (5003, 264), (4099, 777), (700, 4096), (300, 8200)])
def test_head_of_a_few_tokens(tokens, vocab, dim):
    h, w, target = head_inputs(tokens, vocab, dim, seed=11)
    if tokens > 2:
        target[1] = -100
    want = ref.head(h, w, target)
    check_loss(*se().head_loss(h.cuda(), w.cuda(), target.cuda()), want, dim)
    loss, row_loss, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda())
    check_loss(loss, row_loss, want, dim)
    check_grads(dh, dw, want, h, w)


@pytest.mark.parametrize("tokens,vocab,dim", HEADS)
@pytest.mark.parametrize("ignored,dtype", [(0.0, FP), (0.4, BF)])
def test_head_loss_grad(tokens, vocab, dim, ignored, dtype):
    h, w, target = head_inputs(tokens, vocab, dim, seed=1, ignored=ignored)
    out = Guarded((vocab, dim), dtype, fill=3.0)
    loss, row_loss, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda(), dw=out.t)
    want = ref.head(h, w, target)
    check_loss(loss, row_loss, want, dim)
    check_grads(dh, dw, want, h, w)
    assert out.intact()
    again = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda(), dtype=dtype)
    assert torch.equal(again[2], dh) and torch.equal(again[3], dw) and torch.equal(again[1], row_loss)
    only = se().head_loss(h.cuda(), w.cuda(), target.cuda())
    assert torch.equal(only[0], loss) and torch.equal(only[1], row_loss)


def test_head_loss_grad_over_several_pieces():
    # 17000 tokens: a piece buffer holds 7680 of the vocabulary's rows, two pieces
    g = gen(31)
    tokens, vocab, dim = 17000, 9001, 16
    w, h = randn(g, (vocab, dim), BF, 0.5), randn(g, (tokens, dim), BF)
    target = torch.randint(0, vocab, (tokens,), generator=g, dtype=torch.int32)
    target[::3] = -100
    loss, row_loss, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda(), reduction="sum", grad_scale=0.5)
    want = ref.head(h, w, target, mean=False, grad_scale=0.5)
    check_loss(loss, row_loss, want, dim)
    check_grads(dh, dw, want, h, w)


def test_head_loss_grad_over_three_pieces():
    # 6000 tokens: a piece buffer holds 21760 of the vocabulary's rows, the first buffer is used twice
    g = gen(32)
    tokens, vocab, dim = 6000, 47001, 40
    w, h = randn(g, (vocab, dim), BF, 0.3), randn(g, (tokens, dim), BF)
    target = torch.randint(0, vocab, (tokens,), generator=g)
    target[::5] = -100
    before = randn(g, (vocab, dim), FP, 1e-4)
    args = h.cuda(), w.cuda(), target.cuda()
    loss, row_loss, dh, dw = se().head_loss_grad(*args, dw=before.cuda(), accumulate=True)
    want = ref.head(h, w, target)
    check_loss(loss, row_loss, want, dim)
    check_grads(dh, dw, want, h, w, before=before)
    again = se().head_loss_grad(*args, dw=before.cuda(), accumulate=True)
    assert torch.equal(again[2], dh) and torch.equal(again[3], dw)


@pytest.mark.parametrize("dtype", [FP, BF])
@pytest.mark.parametrize("dim", [64, 9])
def test_head_loss_grad_adds_to_a_gradient(dim, dtype):
    h, w, target = head_inputs(50, 400, dim, seed=2, ignored=0.2)
    before = randn(gen(4), (400, dim), dtype, 1e-3)
    loss, row_loss, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda(), dw=before.cuda(), accumulate=True)
    check_grads(dh, dw, ref.head(h, w, target), h, w, before=before)


@pytest.mark.parametrize("tokens", [0, 1, 200])
def test_head_without_any_target(tokens):
    h, w, _ = head_inputs(max(tokens, 1), 300, 64)
    h = h[:tokens]
    target = torch.full((tokens,), 7)
    loss, row_loss, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda(), ignore_index=7)
    assert float(loss) == 0 and row_loss.shape == (tokens,) and bool((row_loss == 0).all())
    assert dh.shape == (tokens, 64) and bool((dh == 0).all()) and bool((dw == 0).all())
    loss, row_loss = se().head_loss(h.cuda(), w.cuda(), target.cuda(), ignore_index=7)
    assert float(loss) == 0


def test_head_targets_outside_the_vocabulary_are_skipped_and_reported():
    import spectral_corrected_optimizer_gb300 as so
    h, w, target = head_inputs(20, 50, 64, seed=3)
    target[4], target[9], target[11] = 50, -1, -100
    loss, row_loss, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda())
    with pytest.raises(so.SpecOptimError, match="target") as e:
        so.check_device()
    assert e.value.code == so.ERR_BOUNDS
    want = ref.head(h, w, target)
    check_loss(loss, row_loss, want, 64)
    check_grads(dh, dw, want, h, w)


def test_head_of_extreme_logits():
    # one logit far above the rest, all logits equal, and logits of the order of 1e4
    w = torch.zeros(600, 16, dtype=BF)
    w[:, 0] = torch.linspace(-1, 1, 600).to(BF)
    h = torch.zeros(4, 16, dtype=BF)
    h[0, 0], h[2, 0], h[3, 0] = 300.0, 1e4, -1e4
    target = torch.tensor([599, 17, 0, 0])
    loss, row_loss, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda())
    want = ref.head(h, w, target)
    check_loss(loss, row_loss, want, 16)
    assert bool(dh.isfinite().all()) and bool(dw.isfinite().all())
    assert abs(float(row_loss[1]) - math.log(600)) < 1e-5


def test_head_keeps_non_finite_rows_visible():
    h, w, target = head_inputs(10, 300, 64, seed=4)
    h[3, 5] = float("nan")
    loss, row_loss = se().head_loss(h.cuda(), w.cuda(), target.cuda())
    assert math.isnan(float(loss)) and bool(row_loss[3].isnan())
    rest = [i for i in range(10) if i != 3]
    assert bool(row_loss[rest].isfinite().all())
    # a token without a target does not count, whatever it holds
    target[3] = -100
    loss, row_loss, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda())
    assert math.isfinite(float(loss)) and bool(dw.isfinite().all()) and bool((dh[3] == 0).all())


def test_head_gradient_against_differences():
    h, w, target = head_inputs(6, 200, 32, seed=5)
    g, step = gen(6), 1e-4
    loss, _, dh, dw = se().head_loss_grad(h.cuda(), w.cuda(), target.cuda())
    f = lambda a, b: float(ref.head(a, b, target)["loss"])  # noqa: E731
    for got, base, which in ((dh, h.double(), 0), (dw, w.double(), 1)):
        u = torch.randn(base.shape, generator=g, dtype=torch.float64)
        args = (lambda d: (base + d * u, w.double())) if which == 0 else (lambda d: (h.double(), base + d * u))
        diff = (f(*args(step)) - f(*args(-step))) / (2 * step)
        # the gradient's own error in norm is below u16; step^2 terms are below 1e-7
        assert abs(diff - float((got.cpu().double() * u).sum())) <= U16 * float(got.cpu().double().norm() * u.norm()) + 1e-6


def test_operators_run_on_another_stream():
    h, w, target = head_inputs(70, 500, 64, seed=7)
    args = [t.cuda() for t in (h, w, target)]
    base = se().head_loss_grad(*args)
    ids, dy = torch.randint(0, 500, (70,), generator=gen(1)).cuda(), h.cuda()
    grad = se().embed_grad(ids, dy, 500)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    got = se().head_loss_grad(*args, stream=st)
    got_grad = se().embed_grad(ids, dy, 500, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(base, got)) and torch.equal(grad, got_grad)


# ---------------------------------------------------------------- offsets beyond 32 bits

FAR = (600_000, 4096)  # 2.46e9 values


def test_embedding_offsets_beyond_32_bits():
    vocab, dim = FAR
    g = gen(12)
    ids = torch.tensor([vocab - 1, 0, vocab - 3, 17]).cuda()
    dy = randn(g, (4, dim), BF).cuda()
    grad = se().embed_grad(ids, dy, vocab, dtype=BF)
    assert torch.equal(grad[ids], dy)
    assert not bool(grad[18:-3].any()) and not bool(grad[-2].any()) and not bool(grad[1:17].any())
    assert torch.equal(se().embed_lookup(grad, ids), dy)


def test_norm_offsets_beyond_32_bits():
    rows, dim = FAR
    x = torch.randn(rows, dim, device="cuda", dtype=BF)
    gamma = randn(gen(13), (dim,), BF).cuda()
    kept, s, y = se().residual_norm(x, None, gamma)
    dx, _, again = se().residual_norm_backward(x, kept, gamma, recompute=True)
    # rows do not depend on one another
    tail = slice(rows - 16, rows)
    kept_t, _, y_t = se().residual_norm(x[tail].clone(), None, gamma)
    dx_t, _, again_t = se().residual_norm_backward(x[tail].clone(), kept_t, gamma, recompute=True)
    for a, b in ((y, y_t), (kept.q.view(torch.uint8), kept_t.q.view(torch.uint8)), (kept.scale, kept_t.scale),
                 (kept.rstd, kept_t.rstd), (dx, dx_t), (again, again_t)):
        assert torch.equal(a[tail], b)


def test_head_offsets_beyond_32_bits():
    vocab, dim = FAR
    g = gen(14)
    w = torch.zeros(vocab, dim, dtype=BF, device="cuda")
    w[-3:] = (0.05 * randn(g, (3, dim))).to(BF).cuda()
    h = randn(g, (3, dim), BF).cuda()
    target = torch.tensor([vocab - 1, vocab - 2, 5])
    loss, row_loss, dh, dw = se().head_loss_grad(h, w, target.cuda(), dtype=BF)
    h64, l = h.double().cpu(), h.double().cpu() @ w[-3:].double().cpu().T
    lse = torch.log(vocab - 3 + l.exp().sum(1))
    want = lse - torch.tensor([l[0, 2], l[1, 1], 0.0], dtype=torch.float64)
    # logits: dim / 16 sums, each cut off by up to 2 u32 of it; the exponentials' sum: fewer than 200 roundings
    off = dim / 16 * 2 * U32 * float(l.abs().max())
    assert bool(((row_loss.cpu().double() - want).abs() <= off + 200 * U32 + 4 * U32 * want.abs()).all())
    d = (l - lse[:, None]).exp()
    d[0, 2] -= 1
    d[1, 1] -= 1
    got, want_dw, mag = dw[-3:].double().cpu(), d.T @ h64 / 3, d.abs().T @ h64.abs() / 3
    # a probability is off by its exponent's error and rounded to 16 bits, as the result is
    assert bool(((got - want_dw).abs() <= (2 * U16 + 2 * off) * mag + U16 * want_dw.abs()).all())
    # row 5 is token 2's target: its own term, and probabilities 1e-6 of the other two
    assert bool(((dw[5].double().cpu() + h64[2] / 3).abs() <= (2 * U16 + 1e-4) * h64.abs().sum(0) / 3).all())
