"""The example that runs the end stages' operators together: its loss falls, and
its first gradients are those of the model written out in float64."""
import os
import sys

import pytest
import torch

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


def test_loss_falls_far_below_the_uniform_guess():
    import train_end_stages as ex
    losses = ex.train(steps=60)
    # ln(1000) = 6.9 is the uniform guess; half of each embedding is masked, yet a token's successor is a fixed function
    assert losses[0] > 6.0 and losses[-1] < 0.5 * losses[0] and min(losses) == min(losses[-20:])


def test_first_gradients_match_float64_autograd():
    import spectral_corrected_optimizer_gb300 as so
    import train_end_stages as ex
    model = ex.EndStages(300, 128, seed=3)
    ids, targets = next(ex.batches(300, 200, 1, seed=4))
    loss = model.micro_batch(ids, targets, step=0, batch_id=0, grad_scale=1.0)
    mask = torch.zeros(200, 128, dtype=torch.float64)
    idx = so.mask_indices(200, 128, model.K, 0, 0, 0).cpu().long()
    mask.scatter_(1, idx, 1.0)
    w = {k: v.cpu().double().requires_grad_() for k, v in model.weights.items()}
    h = w["embed"][ids.cpu()] * mask
    s = h + torch.cat((torch.zeros_like(h[:1]), h[:-1]))
    y = s / torch.sqrt((s * s).mean(-1, keepdim=True) + 1e-5) * w["gamma"]
    want = torch.nn.functional.cross_entropy(y @ w["head"].T, targets.cpu(), ignore_index=ex.IGNORE)
    want.backward()
    want = float(want.detach())
    assert abs(float(loss) - want) <= 2e-2 * want
    for k, g in model.grads.items():
        full = w[k].grad
        # roundings to bf16 (2^-8 each: lookup, sum, y, dy, dx, twice the boundary) and to e4m3 (2^-4) of the
        # norm's input: each is an independent relative error of the values, 2^-4 / sqrt(3) in norm for the largest
        rel = float((g.cpu().double() - full).norm() / full.norm())
        assert rel <= 0.06, (k, rel)
