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
