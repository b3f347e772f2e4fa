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
