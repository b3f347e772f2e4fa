"""The fine-tuning operators at the edges of what their header promises, against the
float64 forms of finetune_ref.py.  Tolerances are those derived in
test_gpu_finetune.py unless a test derives its own."""
import math

import pytest
import torch

import finetune_ref as ref
import test_gpu_finetune as base
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

U16, U32, BF, FP = base.U16, base.U32, base.BF, base.FP
INF = math.inf


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.fixture(autouse=True)
def _clean_flag(_lib):
    yield
    import spectral_corrected_optimizer_gb300 as so
    so.check_device()


# ---------------------------------------------------------------- policy loss

@pytest.mark.parametrize("lengths", [[7, 331, 0, 19], [500, 100, 900] * 40])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_policy_gradient_where_the_divergence_is_only_watched(lengths, reduction):
    # kl_coef 0: the divergence overflows at some tokens, the loss and its gradient are those without a reference
    g = base.gen(len(lengths))
    offsets = base.make_offsets(lengths)
    logp, old, r, a = base.policy_inputs(g, int(offsets[-1]), len(lengths), True)
    r[::5] = logp[::5] + 89.0
    r[1::7] = logp[1::7] + 1e30
    logp[3] = -INF
    args = logp.cuda(), old.cuda(), a.cuda(), offsets.cuda()
    alone = base.ft().policy_loss(*args, reduction=reduction)
    loss, parts, dlogp = base.ft().policy_loss(*args, ref_logp=r.cuda(), reduction=reduction)
    assert bool(dlogp.isfinite().all()) and torch.equal(dlogp, alone[2]) and torch.equal(loss, alone[0])
    assert not bool(parts[1].isfinite()) and torch.equal(parts[::2], alone[1][::2])


@pytest.mark.parametrize("tokens", [1, 3, 700, 50001])
@pytest.mark.parametrize("reduction", ["token", "sum"])
@pytest.mark.parametrize("high", [0.28, INF])
def test_policy_loss_of_tokens_whose_ratio_is_far_from_one(tokens, reduction, high):
    # the gradient of a token is -A r of it, however small r is, and the loss of few tokens has the digits of their r
    g = base.gen(tokens)
    far = torch.exp(torch.rand(tokens, generator=g) * math.log(85.0))  # |d| from 1 to 85
    old = -0.5 * torch.rand(tokens, generator=g)
    up = torch.rand(tokens, generator=g) < 0.25
    logp = torch.where(up, old + far.clamp_max(20.0), old - far)
    a = torch.randn(tokens, generator=g)
    for low, adv in ((0.2, a.abs() + 0.1), (1.0, a)):  # clip_low 1 clips no negative advantage either
        got = base.ft().policy_loss(logp.cuda(), old.cuda(), adv.cuda(), clip_low=low, clip_high=high, reduction=reduction)
        want = ref.policy(logp, old, adv, torch.tensor([0, tokens]), low=low, high=high, reduction=reduction)
        base.check_policy(got, want, 0.0)
        assert torch.equal(got[2].cpu() == 0, want["dlogp"].float() == 0)


def test_policy_loss_of_an_advantage_of_zero_whose_ratio_overflows():
    # nothing is clipped: 0 times the ratio is 0, as it is in 64 bits, and the other tokens keep their gradient
    old = torch.tensor([-100.0, -1.0, -700.0])
    logp, a = torch.tensor([0.0, -1.5, -3.0]), torch.tensor([0.0, 2.0, -0.0])
    loss, parts, dlogp = base.ft().policy_loss(logp.cuda(), old.cuda(), a.cuda(), clip_low=1.0, clip_high=INF)
    want = ref.policy(logp, old, a, torch.tensor([0, 3]), low=1.0, high=INF)
    assert bool(dlogp.isfinite().all()) and dlogp.cpu()[[0, 2]].tolist() == [0.0, 0.0]
    base.check_policy((loss, parts, dlogp), want, 0.0)


@pytest.mark.parametrize("tokens", [100, 5000])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_one_offset_outside_the_tokens_is_reported(tokens, dtype):
    # no sequences: the offset says only where they would begin
    import spectral_corrected_optimizer_gb300 as so
    logp, none = torch.full((tokens,), -1.0).cuda(), torch.empty(0).cuda()
    mask = torch.ones(tokens, dtype=torch.bool).cuda()
    for at in (-5, tokens + 1, 0, tokens):
        offsets = torch.tensor([at], dtype=dtype).cuda()
        for call in (lambda: base.ft().preference_loss(logp, None, offsets),
                     lambda: base.ft().policy_loss(logp, logp, logp, offsets),
                     lambda: base.ft().policy_loss(logp, logp, logp, offsets, mask=mask),
                     lambda: base.ft().policy_loss(logp, logp, none, offsets, reduction="sequence", mask=mask)):
            got = call()
            assert float(got[0]) == 0 and bool((got[-1] == 0).all())
            if 0 <= at <= tokens:
                so.check_device()
                continue
            with pytest.raises(so.SpecOptimError, match="offsets") as e:
                so.check_device()
            assert e.value.code == so.ERR_BOUNDS


# ---------------------------------------------------------------- gradient norm and clipping

def test_clipping_more_tensors_than_a_launch_takes_joins_their_norm_once():
    # each launch would join the partial sums of all of them again: work that grows with the square of the tensors
    import spectral_corrected_optimizer_gb300 as so
    grads = [x.cuda() for x in base.tensors(base.gen(4), [5, 3, 40] * 1100, (FP, BF))]
    before = [x.cpu() for x in grads]
    norm = ref.norm_of(before)
    so.trace_enable(True)
    try:
        so.trace_reset()
        got = base.ft().clip_grads(grads, norm / 2)
        report = so.trace_report()
    finally:
        so.trace_enable(False)
        so.trace_reset()
    assert {k: v[0] for k, v in report.items()} == {"grad_norm": 4, "grad_norm_join": 1, "clip_grads": 4}
    base.inside(got, torch.tensor(norm, dtype=torch.float64), 20 * U32 * norm)
    for x, o in zip(before, grads):
        base.inside(o, x.double() / 2, (base.u_of(o.dtype) + 24 * U32) * x.double().abs() / 2 + 1e-44)


@pytest.mark.parametrize("size,scale", [(1e37, 1.0), (3e33, 1.0), (3e33, -0.5), (1.0, 1e36), (1e-3, 3e38), (1e30, 1e20)])
@pytest.mark.parametrize("most", [1.0, 1e-3, 1e-6])
@pytest.mark.parametrize("norm_type", [2.0, INF])
def test_clipping_by_factors_far_below_what_fp32_holds(size, scale, most, norm_type):
    # max_norm / norm leaves fp32's normal range, the clipped values do not
    x = (torch.randn(20000, generator=base.gen(3)) * size).float()
    x[5] = size * 3
    scale, most = (float(torch.tensor(v)) for v in (scale, most))
    norm = ref.norm_of([x], scale, norm_type)
    want = x.double() * (scale * most / norm)
    for dtype in (FP, BF):
        out = torch.empty_like(x, dtype=dtype, device="cuda")
        got = base.ft().clip_grads([x.cuda()], most, scale=scale, norm_type=norm_type, out=[out])
        if norm < 3.4e38:
            base.inside(got, torch.tensor(norm, dtype=torch.float64), 20 * U32 * norm)
        else:
            assert float(got) == INF
        base.inside(out, want, (base.u_of(dtype) + 24 * U32) * want.abs() + 1e-44)


# ---------------------------------------------------------------- widths and sizes at the borders of the launches' rules

@pytest.mark.parametrize("rows,dim", [(33, 4081), (33, 4083), (33, 4090), (17, 8177), (17, 8178), (17, 8185), (17, 8186)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_layer_norm_of_odd_widths_at_the_borders_of_a_thread_s_pieces(rows, dim, dtype):
    # a row that begins anywhere between two 16-byte boundaries has (dim + 14) / 8 pieces: 512 of them is one for each
    # thread, 1024 two
    base.test_layer_norm_and_its_backward(rows, dim, dtype, True)
    base.test_layer_norm_and_its_backward(rows, dim, dtype, False)


def test_head_logp_backward_of_more_tokens_than_are_listed_by_one_launch():
    # from 65536 tokens on those that take part are counted in stretches first, by target and by gradient
    g = base.gen(5)
    tokens, vocab, dim = 70001, 50, 8
    h, w = base.randn(g, (tokens, dim), BF), base.randn(g, (vocab, dim), BF, 0.5)
    target = torch.randint(0, vocab, (tokens,), generator=g)
    target[::3] = -100
    dlogp = base.randn(g, (tokens,), FP, 1 / tokens)
    dlogp[torch.rand(tokens, generator=g) < 0.3] = 0.0
    _, kept = base.ft().head_logp(h.cuda(), w.cuda(), target.cuda())
    dh, dw = base.ft().head_logp_backward(dlogp.cuda(), kept, h.cuda(), w.cuda(), target.cuda())
    want = base.stage_ends_ref.head(h, w, target, mean=False)
    base.check_weighted(dh, dw, dlogp, want, h, w)


def test_gradients_of_the_norm_s_vectors_over_a_million_rows():
    rows, dim = 1 << 20, 264
    g = torch.Generator("cuda").manual_seed(2)
    x, dy = (torch.empty(rows, dim, dtype=BF, device="cuda").normal_(generator=g) for _ in range(2))
    gamma = torch.ones(dim, dtype=BF, device="cuda")
    kept, s, _ = base.ft().layer_norm(x, None, gamma)
    _, dgamma, dbeta = base.ft().layer_norm_backward(dy, s, kept, gamma)
    sums = torch.zeros(4, dim, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 1 << 16):
        at = slice(i, i + (1 << 16))
        d = dy[at].double()
        n = d * (x[at].double() - kept.mean[at, None].double()) * kept.rstd[at, None].double()
        for k, t in enumerate((n, n.abs(), d, d.abs())):
            sums[k] += t.sum(0)
    # the rows are shared out to at least 152 groups of threads: a column's thread adds at most that share of them, and what
    # the threads leave is added in fewer than 20 steps, the roundings of a term among them
    steps = -(-rows // 152) + 20
    assert bool(((dgamma.double() - sums[0]).abs() <= steps * U32 * sums[1]).all())
    assert bool(((dbeta.double() - sums[2]).abs() <= steps * U32 * sums[3]).all())


def test_losses_of_as_many_tokens_as_a_call_may_have():
    tokens = 1 << 30
    g = torch.Generator("cuda").manual_seed(4)
    logp, old = (torch.empty(tokens, device="cuda").uniform_(-2, 0, generator=g) for _ in range(2))
    a = torch.empty(tokens, device="cuda").normal_(generator=g)
    half = tokens // 2 - 5
    offsets = torch.tensor([3, half, tokens - 1], device="cuda")
    chunks = [slice(i, i + (1 << 26)) for i in range(0, tokens, 1 << 26)]
    at = torch.tensor([0, 2, 3, 4, half - 1, half, half + 1, tokens - 3, tokens - 2, tokens - 1], device="cuda")
    # one pair, scores of half a billion differences each: the sums are kept to 2^-44 and rounded once
    beta = 2.0 ** -12
    loss, pair_loss, rewards, dlogp = base.ft().preference_loss(logp, old, offsets, beta=beta)
    score = torch.stack([sum((logp[s].double() - old[s].double()).sum() for s in [slice(o, min(o + (1 << 26), e)) for o in
                             range(b, e, 1 << 26)]) for b, e in ((3, half), (half, tokens - 1))])
    size = beta * tokens  # |difference| <= 2, and its rounding u32 of it
    base.inside(rewards[0], beta * score.cpu(), U32 * (size + 4 * (beta * score.cpu()).abs()))
    delta = beta * float(score[0] - score[1])
    slope = beta / (1 + math.exp(delta))
    off = 2 * U32 * size  # of delta, and of the slope in parts of 1 / 4 of it
    want = torch.tensor([0, 0, -slope, -slope, -slope, slope, slope, slope, slope, 0], dtype=torch.float64)
    base.inside(dlogp[at], want, (beta * 0.25 * off + 16 * U32 * slope) * (want != 0))
    assert abs(float(loss) - math.log1p(math.exp(-delta))) <= off + 8 * U32 * float(loss)
    del dlogp
    loss, parts, dlogp = base.ft().policy_loss(logp, old, a)
    gain, clipped = 0.0, 0
    for s in chunks:
        d, x = logp[s].double() - old[s].double(), a[s].double()
        far = torch.where(x >= 0, d > math.log1p(0.2), d < math.log1p(-0.2))
        gain += float((x * torch.where(far, torch.where(x >= 0, 1.2, 0.8).double(), torch.exp(d))).sum())
        clipped += int(far.sum())
        slope = torch.where(far, 0.0, -x * torch.exp(d)) / tokens
        assert bool(((dlogp[s].double() - slope).abs() <= 13 * U32 * slope.abs() + 1e-44).all())
    # a thread adds at most 7885 terms of magnitude |a| exp(2) / tokens at most, 13 steps between threads
    steps = (7885 + 13) * U32
    assert abs(float(loss) + gain / tokens) <= steps * math.exp(2) and abs(float(parts[2]) - clipped / tokens) <= steps
