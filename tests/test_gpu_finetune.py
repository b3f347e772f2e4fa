"""GPU parity of the fine-tuning operators (include/finetune.h) with their
definitions in float64 (finetune_ref.py).

u16 = 2^-8 and u32 = 2^-24 are the unit roundoffs of bf16 and fp32.
- LayerNorm: a row's sum runs over at most 72 values in a row, 5 shuffle steps and
  16 warps: 100 u32 of the mean magnitude.  The squares are taken about means m_w
  that are off by that much and of differences that round by u32 max |s|: with
  k = max |s| rstd the variance is off by (100 + 202 k + 2 k + second order) u32, rstd by
  half of it: 150 (1 + k) u32.  y: the differences' error |gamma| rstd 102 u32 max |s|,
  |y - beta| times (that of rstd + 3 u32), 2 u32 of |y - beta| + |beta|, and its rounding.
  Backward: the row sums are such sums, n rounds twice: 110 u32 of the magnitudes of
  dx's terms; dgamma and dbeta add at most `rows` terms: (rows + 20) u32 of them.
- head: as derived in test_gpu_stage_ends.py, d weighted by dlogp.
- preference: each difference rounds once (u32 of its magnitude); their sum is kept to
  2^-40.  delta also rounds to fp32; exp, log1p and a quotient are within 8 u32.
- policy: d = logp - old rounds once, exp is within 4 u32: the ratio is off by
  (|d| + 5) u32 of itself.  q rounds once: exp(q) - 1 is off by u32 |q| exp(q) and 4 u32
  of itself; the divergence by u32 |q| |exp(q) - 1|, 10 u32 of itself, and where it is a
  difference (|q| >= 1/2) u32 (4 |exp(q) - 1| + |q|).  Sums of fp32 terms: 300 u32 of
  their magnitudes (at most 200 terms of a thread, 13 steps between threads).
- norm: at most 32 squares are added in fp32, all else in fp64: 20 u32.  A clipped value
  is off by that, and rounds three times.
"""
import math

import pytest
import torch

import finetune_ref as ref
import stage_ends_ref
import test_gpu_stage_ends as base
from gpu_util import Guarded, ensure_lib

pytestmark = pytest.mark.gpu

U16, U32, BF, FP = base.U16, base.U32, base.BF, base.FP
gen, randn, u_of, shifted = base.gen, base.randn, base.u_of, base.shifted


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.fixture(autouse=True)
def _clean_flag(_lib):
    yield
    import spectral_corrected_optimizer_gb300 as so
    so.check_device()


def ft():
    from spectral_corrected_optimizer_gb300 import finetune
    return finetune


def cuda(t):
    return None if t is None else t.cuda()


def inside(got, want, tol):
    err = (got.cpu().double() - want).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), "off by %.3g of the tolerance" % float((err / (tol + 1e-300)).max())


# ---------------------------------------------------------------- layer norm

NORMS = [(1, 1), (3, 7), (5, 128), (4, 129), (17, 256), (9, 1001), (6, 2048), (3, 4096), (2, 8200), (2, 12345),
         (1, 32768), (700, 264), (2600, 64), (5000, 72), (1300, 33), (40, 8191), (40, 8192), (700, 513), (90, 4104)]


def norm_inputs(rows, dim, dtype, residual, seed=0):
    g = gen(seed + rows * 7 + dim)
    x = (torch.randn(rows, dim, generator=g) + torch.randn(rows, 1, generator=g)) * torch.exp(torch.randn(rows, 1, generator=g))
    x[:, ::97] *= 30
    r = randn(g, (rows, dim), dtype) if residual else None
    gamma, beta = 1 + 0.3 * torch.randn(dim, generator=g), 0.2 * torch.randn(dim, generator=g)
    return x.to(dtype), r, gamma.to(dtype), beta.to(dtype), g


def check_forward(kept, y, s, gamma, beta, eps):
    want_y, mean, rstd = ref.norm_forward(s, gamma, beta, eps)
    top = s.double().abs().amax(-1)
    inside(kept.mean, mean, 100 * U32 * s.double().abs().mean(-1))
    spread = 150 * U32 * (1 + top * rstd)
    inside(kept.rstd, rstd, spread * rstd)
    b = torch.zeros(()) if beta is None else beta.double()
    n = (want_y - b).abs()
    tol = gamma.double().abs() * (rstd * 102 * U32 * top)[:, None] + n * (spread + 3 * U32)[:, None] + 2 * U32 * (n + b.abs())
    inside(y, want_y, tol * (1 + 2 * u_of(y.dtype)) + u_of(y.dtype) * want_y.abs())


def check_backward(dx, dgamma, dbeta, dy, ds, s, kept, gamma):
    w = ref.norm_backward(dy, ds, s, kept.mean.cpu(), kept.rstd.cpu(), gamma)
    rows = dy.shape[0]
    inside(dx, w[0], u_of(dx.dtype) * w[0].abs() + 110 * U32 * w[1])
    inside(dgamma, w[2], (rows + 20) * U32 * w[3])
    if dbeta is not None:
        inside(dbeta, w[4], (rows + 20) * U32 * w[5])


@pytest.mark.parametrize("rows,dim", NORMS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("residual", [True, False])
def test_layer_norm_and_its_backward(rows, dim, dtype, residual):
    x, r, gamma, beta, g = norm_inputs(rows, dim, dtype, residual)
    if not residual and dim % 3 == 0:
        beta = None
    kept, s, y = ft().layer_norm(x.cuda(), cuda(r), gamma.cuda(), cuda(beta), 1e-5)
    want_s = x if r is None else (x.float() + r.float()).to(dtype)
    assert torch.equal(s.cpu(), want_s)
    check_forward(kept, y, want_s, gamma, beta, 1e-5)
    dy = randn(g, (rows, dim), dtype)
    ds = randn(g, (rows, dim), dtype, 0.3) if residual else None
    args = dy.cuda(), s, kept, gamma.cuda()
    dx, dgamma, dbeta = ft().layer_norm_backward(*args, ds=cuda(ds), bias=beta is not None)
    assert (dbeta is None) == (beta is None)
    check_backward(dx, dgamma, dbeta, dy, ds, want_s, kept, gamma)
    again = ft().layer_norm_backward(*args, ds=cuda(ds))
    assert torch.equal(again[0], dx) and torch.equal(again[1], dgamma) and (beta is None or torch.equal(again[2], dbeta))


@pytest.mark.parametrize("rows,dim", [(20000, 72), (9000, 520), (4000, 2048), (3001, 1001)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_layer_norm_of_many_rows(rows, dim, dtype):
    # more rows than groups of threads: every ring turns over several times
    x, r, gamma, beta, g = norm_inputs(rows, dim, dtype, True)
    kept, s, y = ft().layer_norm(x.cuda(), r.cuda(), gamma.cuda(), beta.cuda(), 1e-6)
    check_forward(kept, y, s.cpu(), gamma, beta, 1e-6)
    dy = randn(g, x.shape, dtype)
    check_backward(*ft().layer_norm_backward(dy.cuda(), s, kept, gamma.cuda()), dy, None, s.cpu(), kept, gamma)
    check_backward(*ft().layer_norm_backward(dy.cuda(), s, kept, gamma.cuda(), ds=r.cuda()), dy, r, s.cpu(), kept, gamma)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("rows,dim,by", [(30, 256, 1), (30, 131, 3), (1300, 9, 5), (3, 9001, 2)])
def test_layer_norm_on_unaligned_views(dtype, rows, dim, by):
    x, r, gamma, beta, g = norm_inputs(rows, dim, dtype, True, seed=5)
    kept, s, y = ft().layer_norm(shifted(x, by), shifted(r, 2), shifted(gamma, 1), shifted(beta, 3), 1e-5)
    assert torch.equal(s.cpu(), (x.float() + r.float()).to(dtype))
    check_forward(kept, y, s.cpu(), gamma, beta, 1e-5)
    dy = randn(g, x.shape, dtype)
    got = ft().layer_norm_backward(shifted(dy, 4), shifted(s.cpu(), by), kept, shifted(gamma, 3), ds=shifted(r, by))
    check_backward(*got, dy, r, s.cpu(), kept, gamma)


def test_layer_norm_of_constant_shifted_and_non_finite_rows():
    x = torch.zeros(6, 400)
    x[1] = 7.25                                        # no variance: y is beta
    x[2] = 1e4 + torch.arange(400) * 2.0 ** -6          # a mean that is 2000 times the spread
    x[3, 5] = float("inf")
    x[4, 399] = float("nan")
    x[5] = torch.linspace(-1e18, 1e18, 400)
    gamma, beta = torch.ones(400), torch.linspace(-1, 1, 400)
    kept, s, y = ft().layer_norm(x.cuda(), None, gamma.cuda(), beta.cuda(), 1e-5)
    for row in (0, 1):
        assert torch.equal(y[row].cpu(), beta) and float(kept.mean[row]) == float(x[row, 0])
    good = [0, 1, 2, 5]
    check_forward(ft().NormStatistics(kept.mean[good], kept.rstd[good]), y[good], x[good], gamma, beta, 1e-5)
    assert bool(y[3:5].isnan().all())
    dx, dgamma, dbeta = ft().layer_norm_backward(torch.ones(6, 400).cuda(), s, kept, gamma.cuda())
    assert bool(dx[good].isfinite().all()) and bool(dx[3:5].isnan().all()) and bool((dbeta == 6).all())


def test_layer_norm_of_no_rows():
    gamma, x = torch.ones(64, dtype=BF).cuda(), torch.empty(0, 64, dtype=BF).cuda()
    kept, s, y = ft().layer_norm(x, x, gamma, gamma)
    dx, dgamma, dbeta = ft().layer_norm_backward(x, s, kept, gamma)
    assert y.shape == (0, 64) and dx.shape == (0, 64) and bool((dgamma == 0).all()) and bool((dbeta == 0).all())


def test_layer_norm_backward_against_differences():
    g = gen(21)
    rows, dim, eps, step = 4, 260, 1e-3, 1e-4
    x, dy, u = (torch.randn(rows, dim, generator=g) for _ in range(3))
    gamma, beta = 1 + 0.3 * torch.randn(dim, generator=g), torch.randn(dim, generator=g)
    kept, s, _ = ft().layer_norm(x.cuda(), None, gamma.cuda(), beta.cuda(), eps)
    dx, dgamma, dbeta = ft().layer_norm_backward(dy.cuda(), s, kept, gamma.cuda())
    f = lambda v, c, b: (ref.norm_forward(v, c, b, eps)[0] * dy.double()).sum()  # noqa: E731
    for got, way, at in ((dx, u, 0), (dgamma, u[0], 1), (dbeta, u[1], 2)):
        place = [x.double(), gamma.double(), beta.double()]
        ends = []
        for sign in (1, -1):
            moved = list(place)
            moved[at] = moved[at] + sign * step * way.double()
            ends.append(f(*moved))
        terms = got.cpu().double() * way.double()
        # second-order term of the quotient (step^2) and fp32 sums
        assert abs(float((ends[0] - ends[1]) / (2 * step) - terms.sum())) <= 1e-5 * float(terms.abs().sum())


def test_layer_norm_in_place_through_the_c_entries():
    import spectral_corrected_optimizer_gb300 as so
    for dim in (256, 131):
        x, r, gamma, beta, g = norm_inputs(50, dim, BF, True, seed=3)
        kept, s, y = ft().layer_norm(x.cuda(), r.cuda(), gamma.cuda(), beta.cuda())
        xi, ga, be, y2 = x.cuda(), gamma.cuda(), beta.cuda(), torch.empty_like(y)
        mean, rstd = torch.empty_like(kept.mean), torch.empty_like(kept.rstd)
        p = lambda t: t.data_ptr()  # noqa: E731
        ri, st = r.cuda(), torch.cuda.current_stream().cuda_stream
        so._check(so.lib().layernorm_forward(p(xi), p(ri), p(ga), p(be), 0, 1e-5, p(xi), p(y2), p(mean), p(rstd), 50, dim, st), "f")
        assert torch.equal(xi, s) and torch.equal(y2, y) and torch.equal(mean, kept.mean) and torch.equal(rstd, kept.rstd)
        dy, ds = randn(g, x.shape, BF).cuda(), randn(g, x.shape, BF).cuda()
        want = ft().layer_norm_backward(dy, s, kept, ga, ds=ds)
        for place in (0, 1):
            a = [dy.clone(), ds.clone()]
            dg, db = torch.empty(dim).cuda(), torch.empty(dim).cuda()
            n = so.lib().layernorm_backward_workspace(50, dim)
            ws = torch.empty(n, dtype=torch.uint8).cuda()
            so._check(so.lib().layernorm_backward(p(a[0]), p(a[1]), p(s), p(mean), p(rstd), p(ga), 0, p(a[place]), p(dg), p(db),
                                                  50, dim, p(ws), n, st), "b")
            assert torch.equal(a[place], want[0]) and torch.equal(dg, want[1]) and torch.equal(db, want[2])


def test_layer_norm_writes_only_its_outputs():
    import spectral_corrected_optimizer_gb300 as so
    p = lambda t: t.data_ptr()  # noqa: E731
    st = torch.cuda.current_stream().cuda_stream
    for dtype, code in ((BF, 0), (FP, 1)):
        for rows, dim in ((5, 1001), (9, 64), (3, 2048), (2, 9000)):
            x, r, gamma, beta, g = (t.cuda() if isinstance(t, torch.Tensor) else t for t in norm_inputs(rows, dim, dtype, True))
            s, y, dx = (Guarded((rows, dim), dtype) for _ in range(3))
            mean, rstd, dg, db = Guarded((rows,)), Guarded((rows,)), Guarded((dim,)), Guarded((dim,))
            so._check(so.lib().layernorm_forward(p(x), p(r), p(gamma), p(beta), code, 1e-5, p(s.t), p(y.t), p(mean.t), p(rstd.t),
                                                 rows, dim, st), "f")
            n = so.lib().layernorm_backward_workspace(rows, dim)
            ws = Guarded((n,), torch.uint8)
            so._check(so.lib().layernorm_backward(p(x), p(r), p(s.t), p(mean.t), p(rstd.t), p(gamma), code, p(dx.t), p(dg.t),
                                                  p(db.t), rows, dim, p(ws.t), n, st), "b")
            assert all(b.intact() for b in (s, y, dx, mean, rstd, dg, db, ws)), (dtype, rows, dim)


# ---------------------------------------------------------------- log-probabilities under the head

@pytest.mark.parametrize("tokens,vocab,dim", base.HEADS)
@pytest.mark.parametrize("ignored,dtype", [(0.0, FP), (0.4, BF)])
def test_head_logp_and_its_backward(tokens, vocab, dim, ignored, dtype):
    h, w, target = base.head_inputs(tokens, vocab, dim, seed=1, ignored=ignored)
    want = stage_ends_ref.head(h, w, target, mean=False)
    logp, kept = ft().head_logp(h.cuda(), w.cuda(), target.cuda())
    base.check_loss(-logp.sum(), -logp, want, dim)
    assert torch.equal(-logp, base.se().head_loss(h.cuda(), w.cuda(), target.cuda())[1])
    assert bool((kept[0] == kept[0].round()).all()) and bool((kept[:, ~want["valid"].cuda()] == 0).all())
    dlogp = randn(gen(7), (tokens,)) * torch.exp(3 * randn(gen(8), (tokens,)))
    dlogp[::7] = 0.0
    out = Guarded((vocab, dim), dtype, fill=3.0)
    args = kept, h.cuda(), w.cuda(), target.cuda()
    dh, dw = ft().head_logp_backward(dlogp.cuda(), *args, dw=out.t)
    check_weighted(dh, dw, dlogp, want, h, w)
    assert out.intact()
    again = ft().head_logp_backward(dlogp.cuda(), *args, dtype=dtype)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)


def check_weighted(dh, dw, dlogp, want, h, w, before=None):
    d = -dlogp.double()[:, None] * want["d"]
    e = U16 + base.logit_error(want, h.shape[1])[:, None]
    full_h, full_w = d @ w.double(), d.T @ h.double()
    tol_h, tol_w = e * (d.abs() @ w.double().abs()), (d.abs() * e).T @ h.double().abs()
    if before is not None:
        full_w, tol_w = full_w + before.double(), tol_w + U32 * before.double().abs()
    for got, full, tol in ((dh, full_h, tol_h), (dw, full_w, tol_w)):
        inside(got, full, tol + (U16 if got.dtype == BF else U32) * full.abs() + 1e-30)
        # One token may carry nearly all of the gradient: full = d h then, where each d rounds once (u16 of it, and so of
        # the norm) and the result once more, 2 u16.  Where many tokens share it their roundings add up to less.
        norm = full.norm()
        if norm > 2.0 ** -126:  # below that neither type holds the values
            assert float((got.cpu().double() - full).norm() / norm) <= 2 * U16
    assert bool((dh.cpu()[~(want["valid"] & (dlogp != 0))] == 0).all())


def test_head_logp_backward_over_three_pieces_added_to_a_gradient():
    # 6000 tokens: a piece buffer holds 21760 of the vocabulary's rows, the first buffer is used twice
    g = gen(32)
    tokens, vocab, dim = 6000, 47001, 40
    w, h = randn(g, (vocab, dim), BF, 0.3), randn(g, (tokens, dim), BF)
    target = torch.randint(0, vocab, (tokens,), generator=g, dtype=torch.int32)
    target[:100] = -1
    before, dlogp = randn(g, (vocab, dim), FP, 1e-4), randn(g, (tokens,), FP, 1 / tokens)
    logp, kept = ft().head_logp(h.cuda(), w.cuda(), target.cuda(), ignore_index=-1)
    dh, dw = ft().head_logp_backward(dlogp.cuda(), kept, h.cuda(), w.cuda(), target.cuda(), ignore_index=-1, dw=before.cuda(),
                                     accumulate=True)
    want = stage_ends_ref.head(h, w, target, ignore=-1, mean=False)
    check_weighted(dh, dw, dlogp, want, h, w, before=before)


def test_head_logp_backward_with_nothing_to_do():
    h, w, target = base.head_inputs(40, 300, 64)
    logp, kept = ft().head_logp(h.cuda(), w.cuda(), target.cuda())
    h[3] = float("nan")  # a token whose gradient is 0 has no part, whatever it holds
    dh, dw = ft().head_logp_backward(torch.zeros(40).cuda(), kept, h.cuda(), w.cuda(), target.cuda())
    assert bool((dh == 0).all()) and bool((dw == 0).all())
    none = torch.full((40,), -100)
    logp, kept = ft().head_logp(h.cuda(), w.cuda(), none.cuda())
    dh, dw = ft().head_logp_backward(torch.ones(40).cuda(), kept, h.cuda(), w.cuda(), none.cuda(), dtype=BF)
    assert bool((logp == 0).all()) and bool((dh == 0).all()) and bool((dw == 0).all())
    h, target = h[:0].cuda(), target[:0].cuda()
    logp, kept = ft().head_logp(h, w.cuda(), target)
    dh, dw = ft().head_logp_backward(logp, kept, h, w.cuda(), target)
    assert logp.shape == (0,) and dh.shape == (0, 64) and bool((dw == 0).all())


def test_head_logp_targets_outside_the_vocabulary_are_skipped_and_reported():
    import spectral_corrected_optimizer_gb300 as so
    h, w, target = base.head_inputs(12, 50, 16)
    target[[2, 5]] = torch.tensor([50, -3])
    logp, kept = ft().head_logp(h.cuda(), w.cuda(), target.cuda())
    with pytest.raises(so.SpecOptimError, match="target"):
        so.check_device()
    assert bool((logp[[2, 5]] == 0).all())
    dh, dw = ft().head_logp_backward(torch.ones(12).cuda(), kept, h.cuda(), w.cuda(), target.cuda())
    with pytest.raises(so.SpecOptimError, match="target"):
        so.check_device()
    check_weighted(dh, dw, torch.ones(12), stage_ends_ref.head(h, w, target, mean=False), h, w)


def test_head_logp_backward_against_differences():
    g = gen(3)
    tokens, vocab, dim, step = 9, 40, 32, 2.0 ** -6
    h, w = randn(g, (tokens, dim), BF), randn(g, (vocab, dim), BF, 0.3)
    target, dlogp = torch.randint(0, vocab, (tokens,), generator=g), randn(g, (tokens,))
    _, kept = ft().head_logp(h.cuda(), w.cuda(), target.cuda())
    dh, dw = ft().head_logp_backward(dlogp.cuda(), kept, h.cuda(), w.cuda(), target.cuda())
    u, v = randn(g, (tokens, dim)).double(), randn(g, (vocab, dim)).double()
    f = lambda e: -(dlogp.double() * stage_ends_ref.head(h.double() + e * u, w.double() + e * v, target)["row_loss"]).sum()  # noqa: E731
    # fourth-order quotient; the operators round probabilities and dh to bf16
    diff = (8 * (f(step) - f(-step)) - (f(2 * step) - f(-2 * step))) / (12 * step)
    terms = (dh.cpu().double() * u).sum() + (dw.cpu().double() * v).sum()
    size = (dh.cpu().double() * u).norm() + (dw.cpu().double() * v).norm()
    assert abs(float(diff - terms)) <= 4 * U16 * float(size)


# ---------------------------------------------------------------- preference loss

def make_offsets(lengths, first=0, dtype=torch.int64):
    return torch.cat((torch.tensor([first]), first + torch.cumsum(torch.tensor(lengths, dtype=torch.int64), 0))).to(dtype)


def logps(g, tokens, spread=0.1):
    logp = -torch.randn(tokens, generator=g).square()
    return logp, logp + spread * torch.randn(tokens, generator=g)


def check_preference(got, want, beta):
    loss, pair_loss, rewards, dlogp = got
    size = want["size"]
    inside(rewards, want["rewards"], 1.01 * U32 * (size + 3 * want["rewards"].abs()))
    off = U32 * (1.01 * size.sum(1) + 4 * want["rewards"].abs().sum(1)) + U32 * want["delta"].abs()
    steep = want["slope"].abs() if want["square"] else 1.0
    tol_l = steep * off + 8 * U32 * want["pair_loss"].abs() + (off / beta) ** 2 * want["square"]
    inside(pair_loss, want["pair_loss"], tol_l + 1e-44)
    inside(loss, want["loss"], want["f"] * (tol_l.sum() + len(tol_l) * U32 * want["pair_loss"].abs().sum()) + 1e-44)
    bend = 2 / beta ** 2 if want["square"] else 0.25
    tol_s = 8 * U32 * want["slope_mag"] + bend * off * (not want["hinge"])
    per_token = torch.zeros_like(want["dlogp"])
    for i, s in enumerate(ref.spans(want["offsets"])):
        per_token[s] = tol_s[i // 2] + 6 * U32 * want["slope"][i // 2].abs()
    inside(dlogp, want["dlogp"], per_token * want["factor"].abs() + 1e-44)
    assert bool((dlogp.cpu()[~want["on"]] == 0).all())


def wanted(logp, r, offsets, beta, kind, **more):
    w = ref.preference(logp, r, offsets, beta, kind, **more)
    return {**w, "square": kind == "square", "hinge": kind == "hinge", "offsets": offsets}


LENGTHS = [[1, 1], [45, 45], [0, 3], [3, 0], [0, 0], [7, 200, 1300, 5, 0, 0, 64, 64], [4097, 1023], [9000, 12000],
           [5, 6] * 700, [300, 100] * 200, [40000, 1, 2, 3]]


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("kind,smoothing", [("logistic", 0.0), ("logistic", 0.125), ("hinge", 0.0), ("square", 0.0)])
@pytest.mark.parametrize("average,masked,given,first", [(False, False, True, 0), (True, True, True, 3), (False, True, False, 0),
                                                        (True, False, False, 1)])
def test_preference_loss(lengths, kind, smoothing, average, masked, given, first):
    g = gen(sum(lengths) + len(lengths))
    offsets = make_offsets(lengths, first, torch.int32 if masked else torch.int64)
    tokens = int(offsets[-1]) + first  # some tokens belong to no sequence
    logp, r = logps(g, tokens)
    mask = (torch.rand(tokens, generator=g) < 0.6) if masked else None
    beta = 0.125
    r = r if given else None
    got = ft().preference_loss(logp.cuda(), cuda(r), offsets.cuda(), beta=beta, kind=kind, smoothing=smoothing, average=average,
                               mask=cuda(mask), reduction="sum" if first else "mean", grad_scale=0.5)
    want = wanted(logp, r, offsets, beta, kind, smoothing=smoothing, average=average, mask=mask, mean=not first, grad_scale=0.5)
    if kind == "hinge":  # the inputs stay away from the corner, but for pairs of empty sequences
        assert bool(((want["delta"] - 1).abs() > 1e-4).all())
    check_preference(got, want, beta)
    again = ft().preference_loss(logp.cuda(), cuda(r), offsets.cuda(), beta=beta, kind=kind, smoothing=smoothing, average=average,
                                 mask=cuda(mask), reduction="sum" if first else "mean", grad_scale=0.5)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_preference_loss_ignores_what_does_not_count():
    g = gen(4)
    offsets = make_offsets([30, 50, 20, 9], 5)
    tokens = int(offsets[-1]) + 40
    logp, r = logps(g, tokens)
    mask = torch.rand(tokens, generator=g) < 0.5
    clean = ft().preference_loss(logp.cuda(), r.cuda(), offsets.cuda(), mask=mask.cuda())
    on = ref.counting(offsets, tokens, mask)
    for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(FP).min):
        x, y = (torch.where(on, t, torch.full_like(t, bad)) for t in (logp, r))
        got = ft().preference_loss(x.cuda(), y.cuda(), offsets.cuda(), mask=mask.to(torch.uint8).cuda() * 3)
        assert all(torch.equal(a, b) for a, b in zip(got, clean))


def test_preference_loss_at_extreme_margins():
    # one token a sequence: delta = beta times the difference, exactly
    deltas = torch.tensor([0.0, 1.0, -1.0, 30.0, -30.0, 200.0, -200.0, 3e4, -3e4, float("inf"), -float("inf"), float("nan")])
    logp = torch.stack((deltas, torch.zeros_like(deltas)), 1).view(-1)
    offsets = torch.arange(len(logp) + 1)
    loss, pair_loss, rewards, dlogp = ft().preference_loss(logp.cuda(), None, offsets.cuda(), beta=1.0, reduction="sum")
    d = deltas[:9].double()
    want = torch.nn.functional.softplus(-d, threshold=1e3)
    inside(pair_loss[:9], want, 8 * U32 * want + 1e-44)
    inside(dlogp.view(-1, 2)[:9, 0], -torch.sigmoid(-d), 8 * U32 * torch.sigmoid(-d) + 1e-44)
    assert pair_loss[9:].tolist()[:2] == [0.0, float("inf")] and bool(pair_loss[11].isnan()) and bool(loss.isnan())
    assert dlogp.view(-1, 2)[9:11].tolist() == [[0.0, 0.0], [-1.0, 1.0]] and bool(dlogp[22:].isnan().all())
    hinge = ft().preference_loss(logp.cuda(), None, offsets.cuda(), beta=1.0, kind="hinge", reduction="sum")
    assert hinge[1][:3].tolist() == [1.0, 0.0, 2.0] and hinge[3].view(-1, 2)[:3].tolist() == [[-1, 1], [0, 0], [-1, 1]]
    assert bool(hinge[1][11].isnan())


def test_preference_loss_of_no_pairs_and_long_sums():
    loss, pair_loss, rewards, dlogp = ft().preference_loss(torch.ones(7).cuda(), None, torch.tensor([3]).cuda())
    assert float(loss) == 0 and pair_loss.shape == (0,) and rewards.shape == (0, 2) and bool((dlogp == 0).all())
    # 300000 terms near 100 whose sums differ by little: fp32 sums would be off by 1
    tokens = 300000
    logp = -100 - torch.rand(2 * tokens, generator=gen(2))
    offsets = make_offsets([tokens, tokens])
    got = ft().preference_loss(logp.cuda(), None, offsets.cuda(), beta=2.0 ** -7)
    check_preference(got, wanted(logp, None, offsets, 2.0 ** -7, "logistic"), 2.0 ** -7)
    want = 2.0 ** -7 * logp.double().view(2, -1).sum(1)
    assert bool(((got[2].cpu().double()[0] - want).abs() <= 2 * U32 * want.abs()).all())


def test_preference_loss_gradient_against_differences():
    g = gen(12)
    offsets = make_offsets([30, 20, 15, 40])
    logp, r = logps(g, int(offsets[-1]))
    u, step = torch.randn(len(logp), generator=g).double(), 1e-4
    for kind in ("logistic", "square", "hinge"):
        dlogp = ft().preference_loss(logp.cuda(), r.cuda(), offsets.cuda(), beta=0.25, kind=kind)[3].cpu().double()
        f = lambda e: ref.preference(logp.double() + e * u, r.double(), offsets, 0.25, kind)["loss"]  # noqa: E731
        diff = (f(step) - f(-step)) / (2 * step)
        assert abs(float(diff - (dlogp * u).sum())) <= 1e-5 * float((dlogp * u).abs().sum())


# ---------------------------------------------------------------- policy loss

def check_policy(got, want, kl_coef):
    loss, parts, dlogp = got
    w, q, e, kl = want["weight"], want["q"].abs(), want["e"].abs(), want["kl"]
    tol_gain = want["gain"] * (want["d"].abs() + 6) * U32
    tol_kl = U32 * (q * e + 10 * kl + (q >= 0.5) * (4 * e + q))
    tol_e = U32 * (q * (1 + want["e"]) + 5 * e)
    scale = (want["dlogp"].abs().sum() / (want["slope"].abs() * w).sum().clamp_min(1e-300)) if bool(w.any()) else 1.0
    inside(dlogp, want["dlogp"], scale * w * (~want["clipped"] * tol_gain + abs(kl_coef) * tol_e + 5 * U32 * want["slope"].abs()) + 1e-44)
    assert bool((dlogp.cpu()[~want["on"]] == 0).all())
    tol = [(w * t).sum() + 300 * U32 * (w * m).sum() for t, m in ((tol_gain, want["gain"]), (tol_kl, kl),
                                                                 (0 * kl, want["clipped"].double()))]
    inside(parts, want["parts"], torch.stack(tol) + 1e-44)
    inside(loss, want["loss"], tol[0] + abs(kl_coef) * (tol[1] + 2 * U32 * want["parts"][1]) + 1e-44)


def policy_inputs(g, tokens, count, per_sequence):
    logp = -torch.randn(tokens, generator=g).square()
    old = logp + 0.2 * torch.randn(tokens, generator=g)
    r = logp + 0.5 * torch.randn(tokens, generator=g)
    a = torch.randn(count if per_sequence else tokens, generator=g)
    if len(a):
        a[0] = 0.0
    return logp, old, r, a


@pytest.mark.parametrize("lengths", [[1], [5], [0], [7, 331, 0, 0, 19], [2048] * 3, [20000, 30, 0, 4], [13] * 900, [41000],
                                     [500, 100, 900] * 40, [4096, 4097]])
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("per_sequence,masked,given,first", [(False, False, False, 0), (True, True, True, 0), (False, True, True, 3),
                                                             (True, False, True, 2)])
def test_policy_loss(lengths, reduction, per_sequence, masked, given, first):
    g = gen(sum(lengths) * 3 + len(lengths))
    offsets = make_offsets(lengths, first, torch.int32 if first else torch.int64)
    tokens = int(offsets[-1]) + 2 * first
    logp, old, r, a = policy_inputs(g, tokens, len(lengths), per_sequence)
    mask = (torch.rand(tokens, generator=g) < 0.6) if masked else None
    kl = 0.0625 if given else 0.0
    kwargs = dict(ref_logp=cuda(r) if given else None, mask=cuda(mask), clip_low=0.2, clip_high=0.28, kl_coef=kl,
                  reduction=reduction, grad_scale=0.5, per_sequence=per_sequence)
    got = ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), offsets.cuda(), **kwargs)
    want = ref.policy(logp, old, a, offsets, r if given else None, mask, 0.2, 0.28, kl, reduction, 0.5, per_sequence)
    check_policy(got, want, kl)
    again = ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), offsets.cuda(), **kwargs)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("tokens", [0, 1, 6, 4096, 4097, 70001])
@pytest.mark.parametrize("masked", [True, False])
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
def test_policy_loss_without_sequences(tokens, masked, reduction):
    g = gen(tokens + 5)
    logp, old, r, a = policy_inputs(g, tokens, 1, False)
    mask = (torch.rand(tokens, generator=g) < 0.6) if masked else None
    got = ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), ref_logp=r.cuda(), mask=cuda(mask), kl_coef=0.5, reduction=reduction)
    check_policy(got, ref.policy(logp, old, a, torch.tensor([0, tokens]), r, mask, kl_coef=0.5, reduction=reduction), 0.5)


def test_policy_loss_ignores_what_does_not_count():
    g = gen(14)
    offsets = make_offsets([30, 50, 20], 5)
    tokens = int(offsets[-1]) + 40
    logp, old, r, a = policy_inputs(g, tokens, 3, False)
    mask = torch.rand(tokens, generator=g) < 0.5
    on = ref.counting(offsets, tokens, mask)
    for reduction in ("token", "sequence"):
        kwargs = dict(kl_coef=0.1, reduction=reduction)
        clean = ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), offsets.cuda(), ref_logp=r.cuda(), mask=mask.cuda(), **kwargs)
        for bad in (float("nan"), float("inf"), -float("inf"), torch.finfo(FP).min):
            x, y, z, b = (torch.where(on, t, torch.full_like(t, bad)).cuda() for t in (logp, old, r, a))
            got = ft().policy_loss(x, y, b, offsets.cuda(), ref_logp=z, mask=mask.to(torch.uint8).cuda() * 128, **kwargs)
            assert all(torch.equal(p, q) for p, q in zip(got, clean))


def test_policy_loss_with_nothing_that_counts():
    logp = torch.zeros(90).cuda()
    offsets = make_offsets([40, 50]).cuda()
    mask = torch.zeros(90, dtype=torch.bool).cuda()
    for reduction in ("token", "sequence", "sum"):
        loss, parts, dlogp = ft().policy_loss(logp, logp, logp, offsets, mask=mask, reduction=reduction)
        assert float(loss) == 0 and bool((parts == 0).all()) and bool((dlogp == 0).all())
    loss, parts, dlogp = ft().policy_loss(logp, logp, logp, torch.tensor([50]).cuda(), per_sequence=False)
    assert float(loss) == 0 and bool((dlogp == 0).all())
    mask[40:] = True  # a sequence without a token that counts adds 0 to the mean of two
    loss, parts, _ = ft().policy_loss(logp, logp, torch.ones(2).cuda(), offsets, mask=mask, reduction="sequence")
    assert float(loss) == -0.5


def test_policy_loss_clips_at_the_bound_in_more_than_fp32():
    # logp - old lies a little beside log(1 + high) and log(1 - low): fp32's ratio is the bound on both sides
    high, low = 0.28, 0.2
    edge = torch.tensor([math.log(1 + high)] * 3 + [math.log(1 - low)] * 3, dtype=torch.float64)
    old = torch.full((6,), -3.0)
    near = torch.tensor([-1, 0, 1] * 2)
    logp = (edge + old.double()).float()
    step = torch.where(near > 0, torch.nextafter(logp, torch.full_like(logp, 9.0)), torch.nextafter(logp, torch.full_like(logp, -9.0)))
    logp = torch.where(near == 0, logp, step)
    a = torch.tensor([1.0] * 3 + [-1.0] * 3)
    want = ref.policy(logp, old, a, torch.tensor([0, 6]), low=low, high=high)
    assert 0 < int(want["clipped"].sum()) < 6
    loss, parts, dlogp = ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), clip_low=low, clip_high=high)
    assert torch.equal(dlogp.cpu() == 0, want["clipped"])
    # a million pairs at random distances of the last places
    g = gen(6)
    old = -8 * torch.rand(1 << 20, generator=g)
    logp = (old.double() + math.log(1 + high)).float()
    a = torch.ones(1 << 20)
    want = ref.policy(logp, old, a, torch.tensor([0, 1 << 20]), low=low, high=high)
    dlogp = ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), clip_low=low, clip_high=high)[2]
    assert 1000 < int(want["clipped"].sum()) < (1 << 20) - 1000 and torch.equal(dlogp.cpu() == 0, want["clipped"])


def test_policy_loss_at_extreme_ratios():
    inf = float("inf")
    logp = torch.tensor([0.0, 0.0, -200.0, -200.0, 0.0, 0.0, 0.0])
    old = torch.tensor([-200.0, -200.0, 0.0, 0.0, -inf, -inf, -inf])
    a = torch.tensor([1.0, -1.0, 1.0, -1.0, 2.0, -1.0, 0.0])
    got = [ft().policy_loss(logp[i:i + 1].cuda(), old[i:i + 1].cuda(), a[i:i + 1].cuda(), clip_low=0.5, clip_high=0.25)
           for i in range(7)]
    assert [float(x[0]) for x in got] == [-1.25, inf, 0.0, 0.5, -2.5, inf, -0.0]
    assert [float(x[2]) for x in got] == [0.0, inf, 0.0, 0.0, 0.0, inf, 0.0]
    assert [float(x[1][2]) for x in got] == [1.0, 0.0, 0.0, 1.0, 1.0, 0.0, 1.0]
    # clip_low 1 and an infinite clip_high never clip
    x = ft().policy_loss(logp[:4].cuda(), (logp[:4] + 1).cuda(), a[:4].cuda(), clip_low=1.0, clip_high=inf)
    assert float(x[1][2]) == 0


def test_policy_loss_gradient_against_differences():
    g = gen(17)
    offsets = make_offsets([30, 20, 1, 40])
    tokens = int(offsets[-1])
    logp, old, r, a = policy_inputs(g, tokens, 4, True)
    mask, u, step = torch.rand(tokens, generator=g) < 0.7, torch.randn(tokens, generator=g).double(), 1e-6
    for reduction in ("token", "sequence"):
        dlogp = ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), offsets.cuda(), ref_logp=r.cuda(), mask=mask.cuda(), kl_coef=0.5,
                                 reduction=reduction)[2].cpu().double()
        f = lambda e: ref.policy(logp.double() + e * u, old.double(), a, offsets, r.double(), mask, 0.2, 0.2, 0.5, reduction,  # noqa: E731
                                 per_sequence=True)["loss"]
        diff = (f(step) - f(-step)) / (2 * step)
        assert abs(float(diff - (dlogp * u).sum())) <= 1e-5 * float((dlogp * u).abs().sum())


@pytest.mark.parametrize("by", [1, 2, 3])
def test_losses_on_unaligned_views(by):
    g = gen(by)
    offsets = make_offsets([50, 70, 9, 300], 2)
    tokens = int(offsets[-1]) + 5
    logp, old, r, a = policy_inputs(g, tokens, 4, False)
    mask = torch.rand(tokens, generator=g) < 0.7
    args = shifted(logp, by), shifted(r, 2), shifted(offsets, 1)
    got = ft().preference_loss(*args, mask=shifted(mask, by))
    check_preference(got, wanted(logp, r, offsets, float(torch.tensor(0.1)), "logistic", mask=mask), 0.1)
    got = ft().policy_loss(shifted(logp, by), shifted(old, 1), shifted(a, 3), shifted(offsets, 1), ref_logp=shifted(r, by),
                           mask=shifted(mask, by), kl_coef=0.5)
    check_policy(got, ref.policy(logp, old, a, offsets, r, mask, kl_coef=0.5), 0.5)


def test_offsets_that_break_the_rule_are_reported_and_stay_within_the_tokens():
    import spectral_corrected_optimizer_gb300 as so
    tokens = 100
    logp = Guarded((tokens,), fill=-1.0)
    for bad in ([0, 40, 101], [-1, 40, 100], [0, 60, 50], [0, 2 ** 40, 100], [100, 50, 0]):
        offsets = torch.tensor(bad).cuda()
        for call in (lambda: ft().preference_loss(logp.t, None, offsets),
                     lambda: ft().policy_loss(logp.t, logp.t, torch.ones(2).cuda(), offsets),
                     lambda: ft().policy_loss(logp.t, logp.t, torch.ones(2).cuda(), offsets, reduction="sequence",
                                              mask=torch.ones(tokens, dtype=torch.bool).cuda())):
            call()
            with pytest.raises(so.SpecOptimError, match="offsets") as e:
                so.check_device()
            assert e.value.code == so.ERR_BOUNDS and logp.intact()


# ---------------------------------------------------------------- gradient norm and clipping

def tensors(g, sizes, dtypes, spread=2.0):
    return [randn(g, (n,), dtypes[i % len(dtypes)], math.exp(spread * float(torch.randn((), generator=g))))
            for i, n in enumerate(sizes)]


SIZES = [[1], [0], [], [7, 0, 3], [8192], [8193, 1, 8191], [100000, 33, 5, 70001], [17] * 63, [17] * 64, [17] * 65, [1000] * 300,
         [3] * 1500, [40000] * 1100, [5_000_001, 12, 3_000_000]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dtypes", [(FP,), (BF,), (BF, FP, FP)])
@pytest.mark.parametrize("norm_type", [2.0, math.inf])
def test_grad_norm_and_clipping(sizes, dtypes, norm_type):
    g = gen(sum(sizes) + len(sizes))
    grads = tensors(g, sizes, dtypes)
    for scale in (1.0, -0.25):
        norm = ref.norm_of(grads, scale, norm_type)
        got = ft().grad_norm([x.cuda() for x in grads], scale=scale, norm_type=norm_type)
        inside(got, torch.tensor(norm, dtype=torch.float64), 20 * U32 * norm)
        for most in (norm * 0.5, norm * 1.5 + 1e-3):
            factor = scale * min(1.0, most / norm if norm else 1.0)
            # into other tensors of the other type, then in place
            device = [x.cuda() for x in grads]
            outs = [Guarded((n,), FP if x.dtype == BF else BF) for n, x in zip(sizes[:40], grads)]
            outs_t = [o.t for o in outs] + [torch.empty_like(x) for x in device[40:]]
            got_norm = ft().clip_grads(device, most, scale=scale, norm_type=norm_type, out=outs_t)
            assert torch.equal(got_norm, got) and all(o.intact() for o in outs)
            assert all(torch.equal(a.cpu(), b) for a, b in zip(device, grads))
            ft().clip_grads(device, most, scale=scale, norm_type=norm_type)
            for results in (outs_t, device):
                for x, o in zip(grads, results):
                    want = x.double() * factor
                    inside(o, want, (u_of(o.dtype) + 24 * U32) * want.abs() + 1e-44)


def test_clipping_leaves_gradients_within_the_limit_alone():
    g = gen(2)
    grads = [x.cuda() for x in tensors(g, [1000, 70000, 3], (FP, BF))]
    before = [x.clone() for x in grads]
    norm = ft().clip_grads(grads, float("inf"))
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    again = ft().clip_grads(grads, float(norm))  # at the limit
    assert torch.equal(again, norm) and all(torch.equal(a, b) for a, b in zip(grads, before))
    ft().clip_grads(grads, 0.0)
    assert all(bool((x == 0).all()) for x in grads)
    assert float(ft().clip_grads(grads, 1.0)) == 0 and all(bool((x == 0).all()) for x in grads)


@pytest.mark.parametrize("size", [1e-42, 1e-30, 1e-22, 1e-18, 1e15, 1e18, 1e25, 1e37])
def test_grad_norm_over_the_whole_range(size):
    x = (torch.randn(20000, generator=gen(3)) * size).float()
    x[5] = size * 3
    want = ref.norm_of([x])
    got = ft().grad_norm([x.cuda(), torch.zeros(50).cuda()])
    if want < 3.4e38:
        inside(got, torch.tensor(want, dtype=torch.float64), 20 * U32 * want + 1e-45)
    else:  # infinite in fp32, but not where the values are scaled by it
        assert float(got) == math.inf
    y, most = x.cuda(), min(want / 8, 2.0 ** 127)
    ft().clip_grads([y], most)
    most = float(torch.tensor(most))
    inside(y, x.double() * (most / want), 24 * U32 * x.double().abs() * (most / want) + 2e-45)


def test_clipping_values_that_are_not_finite():
    x = torch.randn(9000, generator=gen(3)).cuda()
    y = x.clone()
    y[8500] = float("inf")
    for kind in (2.0, math.inf):
        a, b = x.clone(), y.clone()
        assert float(ft().clip_grads([a, b], 1.0, norm_type=kind)) == math.inf
        assert bool((a == 0).all()) and bool(b[8500].isnan()) and int(b.isnan().sum()) == 1
        b[8500] = float("nan")
        a = x.clone()
        assert bool(ft().clip_grads([a, b], 1.0, norm_type=kind).isnan()) and bool(a.isnan().all()) and bool(b.isnan().all())
        assert bool(ft().grad_norm([x, b], norm_type=kind).isnan())


@pytest.mark.parametrize("din,dout", [(BF, BF), (FP, FP), (BF, FP), (FP, BF)])
def test_clipping_unaligned_views(din, dout):
    g = gen(9)
    grads = tensors(g, [9001, 300, 20000], (din,))
    device = [shifted(x, k) for x, k in zip(grads, (1, 3, 0))]
    outs = [shifted(torch.zeros_like(x, dtype=dout), k) for x, k in zip(grads, (5, 0, 1))]
    norm = ref.norm_of(grads)
    got = ft().clip_grads(device, norm / 3, out=outs)
    inside(got, torch.tensor(norm, dtype=torch.float64), 20 * U32 * norm)
    for x, o in zip(grads, outs):
        want = x.double() / 3
        inside(o, want, (u_of(dout) + 24 * U32) * want.abs())


def test_clipping_refuses_tensors_that_overlap():
    import spectral_corrected_optimizer_gb300 as so
    flat = torch.ones(1000).cuda()
    other = torch.ones(1000).cuda()
    for grads, out in (([flat, flat], None), ([flat[:600], flat[500:]], None), ([flat, other], [other, flat]),
                       ([flat[:500]], [flat[1:501]]), ([flat[:500]], [flat[:500].view(BF)[:500]]),
                       ([flat, other], [torch.empty(1000).cuda()] * 2)):
        with pytest.raises(so.SpecOptimError, match="overlap") as e:
            ft().clip_grads(grads, 1.0, out=out)
        assert e.value.code == so.ERR_INVALID_ARG
    assert bool((flat == 1).all()) and bool((other == 1).all())
    # reading the same tensor twice is a norm like any other; neighbours in one buffer do not overlap
    assert abs(float(ft().grad_norm([flat, flat])) - 2000 ** 0.5) < 1e-4
    ft().clip_grads(list(flat.split([400, 600])), 1.0)
    assert abs(float(ft().grad_norm([flat])) - 1) < 1e-6


# ---------------------------------------------------------------- more than one round of a launch's blocks, large tensors

@pytest.mark.parametrize("lengths", [[5, 6, 0, 9] * 6000, [600, 500] * 1500])
def test_preference_loss_of_many_pairs(lengths):
    # more pairs than a launch has blocks, and more slices than the GPU holds
    g = gen(len(lengths))
    offsets = make_offsets(lengths)
    tokens = int(offsets[-1])
    logp, r = logps(g, tokens)
    mask = torch.rand(tokens, generator=g) < 0.8
    got = ft().preference_loss(logp.cuda(), r.cuda(), offsets.cuda(), beta=0.125, mask=mask.cuda())
    check_preference(got, wanted(logp, r, offsets, 0.125, "logistic", mask=mask), 0.125)


@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("lengths,per_sequence", [([90, 3, 0, 150, 7] * 1200, True), ([900, 40, 0, 1500] * 400, True),
                                                  ([900, 40, 0, 1500] * 400, False)])
def test_policy_loss_of_many_sequences(lengths, per_sequence, reduction):
    # more sequences than the first launch has blocks, more tiles than the second one
    g = gen(len(lengths))
    offsets = make_offsets(lengths, 2)
    tokens = int(offsets[-1]) + 700
    logp, old, r, a = policy_inputs(g, tokens, len(lengths), per_sequence)
    mask = torch.rand(tokens, generator=g) < 0.8
    kwargs = dict(kl_coef=0.0625, reduction=reduction, per_sequence=per_sequence)
    got = ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), offsets.cuda(), ref_logp=r.cuda(), mask=mask.cuda(), **kwargs)
    check_policy(got, ref.policy(logp, old, a, offsets, r, mask, **kwargs), 0.0625)


def test_operators_on_more_than_2_to_the_31_values():
    rows, dim = 1 << 20, 2056
    x = torch.empty(rows, dim, dtype=BF, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    gamma = torch.ones(dim, dtype=BF, device="cuda")
    kept, s, y = ft().layer_norm(x, None, gamma, gamma)
    pick = torch.tensor([0, 1, rows // 2, rows - 3, rows - 1], device="cuda")
    stats = ft().NormStatistics(kept.mean[pick], kept.rstd[pick])
    check_forward(stats, y[pick], x[pick].cpu(), gamma.cpu(), gamma.cpu(), 1e-5)
    dx, dgamma, dbeta = ft().layer_norm_backward(y, x, kept, gamma, ds=x)
    w = ref.norm_backward(y[pick].cpu(), x[pick].cpu(), x[pick].cpu(), stats.mean.cpu(), stats.rstd.cpu(), gamma.cpu())
    inside(dx[pick], w[0], U16 * w[0].abs() + 110 * U32 * w[1])
    # y = n + 1: dbeta is the number of rows, and so is dgamma, up to the statistics of a million normal values
    assert bool(((dbeta / rows - 1).abs() < 0.01).all()) and bool(((dgamma / rows - 1).abs() < 0.02).all())
    del dx, y
    want = float(torch.sqrt(sum((c.double() ** 2).sum() for c in x.split(1 << 17))))
    flat = x.view(-1)
    before = flat[-5:].clone()
    norm = ft().clip_grads([flat[:7], flat[7:]], want / 2)
    assert abs(float(norm) / want - 1) <= 20 * U32
    assert bool(((flat[-5:].double() - before.double() / 2).abs() <= (U16 + 24 * U32) * before.double().abs() / 2).all())
    assert abs(float(ft().grad_norm([flat])) / want * 2 - 1) <= U16


# ---------------------------------------------------------------- streams, graphs, together

def step_inputs(seed=0):
    g = gen(seed)
    tokens, vocab, dim = 240, 700, 72
    x, r, gamma, beta, _ = norm_inputs(tokens, dim, BF, True, seed)
    w = randn(g, (vocab, dim), BF, 0.1)
    target = torch.randint(0, vocab, (tokens,), generator=g)
    target[::5] = -100
    offsets = make_offsets([70, 50, 60, 60])
    ref_logp = -torch.rand(tokens, generator=g) * 8
    return [t.cuda() for t in (x, r, gamma, beta, w, target, offsets, ref_logp)]


def fine_tuning_step(x, r, gamma, beta, w, target, offsets, ref_logp):
    f = ft()
    stats, s, y = f.layer_norm(x, r, gamma, beta)
    logp, kept = f.head_logp(y, w, target)
    loss, pair_loss, rewards, dlogp = f.preference_loss(logp, ref_logp, offsets, mask=target != -100)
    dy, dw = f.head_logp_backward(dlogp, kept, y, w, target)
    dx, dgamma, dbeta = f.layer_norm_backward(dy, s, stats, gamma)
    norm = f.clip_grads([dw, dgamma, dbeta], 1e-3)
    return loss, rewards, dx, dw, dgamma, dbeta, norm


def test_a_step_of_all_operators_against_autograd_in_64_bits():
    args = step_inputs()
    loss, rewards, dx, dw, dgamma, dbeta, norm = fine_tuning_step(*args)
    x, r, gamma, beta, w, target, offsets, ref_logp = (t.cpu() for t in args)
    s = (x.float() + r.float()).to(BF).double().requires_grad_()
    w64, g64, b64 = (t.double().requires_grad_() for t in (w, gamma, beta))
    y = torch.nn.functional.layer_norm(s, (72,), g64, b64, 1e-5)
    logits = y @ w64.T
    on = target != -100
    logp = torch.log_softmax(logits, 1).gather(1, target.clamp_min(0)[:, None])[:, 0]
    d = torch.where(on, logp - ref_logp.double(), torch.zeros(())).double()
    score = torch.stack([d[v].sum() for v in ref.spans(offsets)]).view(-1, 2) * 0.1
    total = -torch.nn.functional.logsigmoid(score[:, 0] - score[:, 1]).mean()
    total.backward()
    full = math.sqrt(sum(float((t.grad ** 2).sum()) for t in (w64, g64, b64)))
    c = min(1.0, 1e-3 / full)
    # y, the probabilities and dh round to bf16 on the way
    rel = lambda a, b: float((a.cpu().double() - b).norm() / b.norm())  # noqa: E731
    total = float(total.detach())
    assert abs(float(loss) - total) <= 0.01 * abs(total)
    assert rel(rewards, score.detach()) <= 2 * U16
    assert abs(float(norm) / full - 1) <= 2 * U16
    for got, want in ((dx, s.grad), (dw, w64.grad * c), (dgamma, g64.grad * c), (dbeta, b64.grad * c)):
        assert rel(got, want) <= 4 * U16


def test_a_step_on_another_stream_and_replayed_from_graphs():
    args, others = step_inputs(), step_inputs(3)
    want, want_others = fine_tuning_step(*args), fine_tuning_step(*others)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fine_tuning_step(*args)
    stats, s, y = ft().layer_norm(*args[:4], stream=side)
    norm = ft().grad_norm([s, y], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(norm, ft().grad_norm([s, y]))
    # two captured graphs, replayed in turn and on inputs that changed
    graphs = []
    for inputs in (args, others):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fine_tuning_step(*inputs)
        graphs.append((graph, out))
    for _ in range(2):
        for (graph, out), w in zip(graphs, (want, want_others)):
            graph.replay()
    for (graph, out), w in zip(graphs, (want, want_others)):
        assert all(torch.equal(a, b) for a, b in zip(out, w))
    for mine, new in zip(args, others):
        mine.copy_(new)
    graphs[0][0].replay()
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], want_others))
    graph, inputs = torch.cuda.CUDAGraph(), step_inputs()
    a = torch.randn(240, generator=gen(1)).cuda()
    call = lambda: ft().policy_loss(inputs[7], a * 0 - 3, a, inputs[6], ref_logp=inputs[7] * 0.9, mask=inputs[5] != -100, kl_coef=0.1)  # noqa: E731
    want = call()
    with torch.cuda.graph(graph):
        out = call()
    graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(out, want))
