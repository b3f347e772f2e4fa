"""The fine-tuning example (examples/train_preference.py) runs, and its gradients are those of the model written out in
float64 with autograd.  x, s, y, dy, ds and dx are rounded to bf16 on the way (2^-8 each at most, partly shared): a
gradient that passes through all of them is held to 6 of these in norm, the head's and the norm's to 4."""
import os
import sys

import pytest
import torch

from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U16 = 2.0 ** -8


@pytest.fixture(scope="module")
def example():
    ensure_lib()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import train_preference
    return train_preference


def reference(model, batch):
    """float64 copies of the weights that require gradients, and logp from them."""
    w = {k: v.cpu().double().requires_grad_() for k, v in model.weights.items()}
    rounded = {k: w[k] + (w[k].detach().float().bfloat16().double() - w[k].detach()) for k in w}
    ids, targets = batch.ids.cpu(), batch.targets.cpu()
    x = rounded["embed"][ids]
    s = x + torch.cat((torch.zeros_like(x[:1]), x[:-1]))
    s = s + (s.detach().bfloat16().double() - s.detach())
    y = torch.nn.functional.layer_norm(s, (model.dim,), rounded["gamma"], rounded["beta"], 1e-5)
    logp = torch.log_softmax(y @ rounded["head"].T, 1).gather(1, targets.clamp_min(0)[:, None])[:, 0]
    return w, torch.where(targets != -100, logp, torch.zeros_like(logp))


def compare(model, w, loss, want):
    want.backward()
    assert abs(float(loss) - float(want.detach())) <= 0.02 * abs(float(want.detach())) + 1e-3
    for k, bound in (("head", 4), ("gamma", 4), ("beta", 4), ("embed", 6)):
        got, full = model.grads[k].cpu().double(), w[k].grad
        assert float((got - full).norm() / full.norm()) <= bound * U16, k


def spans(batch):
    o = batch.offsets.tolist()
    return [slice(a, b) for a, b in zip(o[:-1], o[1:])]


def setup(example, seed):
    model, start = example.Model(300, 72), example.Model(300, 72, seed=5)
    batch = example.make_batch(300, 12, 20, seed)
    batch.ref_logp, _ = start.forward(batch)
    return model, batch


def test_preference_gradients(example):
    model, batch = setup(example, 1)
    loss, rewards = model.preference(batch, beta=0.25)
    w, logp = reference(model, batch)
    d = logp - batch.ref_logp.cpu().double()
    score = 0.25 * torch.stack([(d * batch.mask.cpu())[s].sum() for s in spans(batch)]).view(-1, 2)
    compare(model, w, loss, -torch.nn.functional.logsigmoid(score[:, 0] - score[:, 1]).mean())


def test_policy_gradients(example):
    model, batch = setup(example, 2)
    advantages = torch.randn(24, generator=torch.Generator().manual_seed(3))
    old, _ = model.forward(batch)
    old = old + 0.02  # every ratio is near exp(-0.02): none is clipped, in either precision
    loss, parts = model.policy(batch, advantages.cuda(), old, kl_coef=0.05)
    w, logp = reference(model, batch)
    mask = batch.mask.cpu()
    q = batch.ref_logp.cpu().double() - logp
    total = 0
    # the ratio is taken at the kernel's own log-probabilities: bf16 moves them by more than the ratio's distance from 1
    own = model.forward(batch)[0].cpu().double()
    ratio = torch.exp(own - old.cpu().double()) * torch.exp(logp - logp.detach())
    for i, s in enumerate(spans(batch)):
        per = -advantages[i].double() * ratio[s] + 0.05 * (torch.expm1(q[s]) - q[s])
        total = total + (per * mask[s]).sum() / mask[s].sum() / 24
    assert float(parts[2]) == 0
    compare(model, w, loss, total)


def test_training_runs_and_clips(example):
    seen = example.train(steps=6, vocab=200, dim=64, pairs=8)
    assert len(seen) == 6 and all(torch.tensor(seen).isfinite().flatten())
    model, batch = setup(example, 4)
    model.preference(batch)
    before = {k: v.clone() for k, v in model.grads.items()}
    norm = float(torch.sqrt(sum((v.double() ** 2).sum() for v in before.values())))
    weights = {k: v.clone() for k, v in model.weights.items()}
    assert abs(float(model.step(0.01, max_norm=norm / 4)) / norm - 1) <= 20 * 2.0 ** -24
    assert all(bool((v == 0).all()) for v in model.grads.values())
    # AdamW's first step is lr times the sign of the gradient, however it was scaled
    for k, v in before.items():
        moved = weights[k] - model.weights[k]
        large = v.abs() > 1e-4
        assert bool(((moved - 0.01 * v.sign())[large].abs() <= 1e-5 + 1e-6 * weights[k][large].abs()).all()), k
