"""Fine-tunes a toy language model on pairs of answers, on one GPU: the operators of a fine-tuning step together.

  x = E[id],  s = x + (the row in front of it),  y = LayerNorm(s) gamma + beta,
  logp = log-probability of each answer token under softmax(y W^T),
  loss = preference of the chosen answer over the other one, against the frozen start,
         or the clipped policy loss with a KL term towards it

The backward pass mirrors it: the loss gives its gradient in the log-probabilities, head_logp_backward turns it into
dL/dy and adds dL/dW, layer_norm_backward gives dL/ds, dL/dgamma and dL/dbeta, embed_grad adds up dL/dE; all gradients
are clipped by their global norm and the framework's AdamW steps the fp32 weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spectral_corrected_optimizer_gb300 as so  # noqa: E402
from spectral_corrected_optimizer_gb300 import finetune as ft  # noqa: E402
from spectral_corrected_optimizer_gb300 import stage_ends as se  # noqa: E402

IGNORE = -100


class Batch:
    """Packed sequences: token ids, their successors (IGNORE within prompts and behind the end), where each begins, and
    what the frozen start says of them."""

    def __init__(self, ids, targets, offsets):
        self.ids, self.targets, self.offsets = ids, targets, offsets
        self.mask = targets != IGNORE
        self.ref_logp = None


class Model:
    """Weights, gradients and AdamW state."""

    def __init__(self, vocab: int, dim: int, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.dim = vocab, dim
        self.weights = {"embed": torch.randn(vocab, dim, generator=g, device="cuda"),
                        "gamma": torch.ones(dim, device="cuda"), "beta": torch.zeros(dim, device="cuda"),
                        "head": torch.randn(vocab, dim, generator=g, device="cuda") * dim ** -0.5}
        self.grads = {k: torch.zeros_like(w) for k, w in self.weights.items()}
        self.moments = {k: (torch.zeros_like(w), torch.zeros_like(w)) for k, w in self.weights.items()}
        self.t = 0

    def forward(self, batch):
        """(logp, what the backward pass needs)."""
        gamma, beta, head = (self.weights[k].bfloat16() for k in ("gamma", "beta", "head"))
        x = se.embed_lookup(self.weights["embed"], batch.ids, dtype=torch.bfloat16)
        before = torch.cat((torch.zeros_like(x[:1]), x[:-1]))
        stats, s, y = ft.layer_norm(x, before, gamma, beta)
        logp, kept = ft.head_logp(y, head, batch.targets, ignore_index=IGNORE)
        return logp, (gamma, head, stats, s, y, kept)

    def backward(self, batch, dlogp, state):
        """Adds the gradients of a loss with gradient dlogp to self.grads."""
        gamma, head, stats, s, y, kept = state
        dy, _ = ft.head_logp_backward(dlogp, kept, y, head, batch.targets, ignore_index=IGNORE, dw=self.grads["head"],
                                      accumulate=True)
        ds, dgamma, dbeta = ft.layer_norm_backward(dy, s, stats, gamma)
        self.grads["gamma"] += dgamma
        self.grads["beta"] += dbeta
        dx = ds + torch.cat((ds[1:], torch.zeros_like(ds[:1])))
        se.embed_grad(batch.ids, dx, self.vocab, out=self.grads["embed"], accumulate=True)

    def preference(self, batch, beta: float = 0.5, grad_scale: float = 1.0):
        """(loss, rewards) of the pairs 2p over 2p + 1; their gradients are added to self.grads."""
        logp, state = self.forward(batch)
        loss, _, rewards, dlogp = ft.preference_loss(logp, batch.ref_logp, batch.offsets, beta=beta, mask=batch.mask,
                                                     grad_scale=grad_scale)
        self.backward(batch, dlogp, state)
        return loss, rewards

    def policy(self, batch, advantages, old_logp, kl_coef: float = 0.05, grad_scale: float = 1.0):
        """(loss, parts) of rollouts with one advantage each; their gradients are added to self.grads."""
        logp, state = self.forward(batch)
        loss, parts, dlogp = ft.policy_loss(logp, old_logp, advantages, batch.offsets, ref_logp=batch.ref_logp,
                                            mask=batch.mask, kl_coef=kl_coef, reduction="sequence", grad_scale=grad_scale,
                                            per_sequence=True)
        self.backward(batch, dlogp, state)
        return loss, parts

    def step(self, lr: float, max_norm: float = 1.0):
        """One AdamW step on the clipped gradients; the norm that they had."""
        self.t += 1
        norm = ft.clip_grads(list(self.grads.values()), max_norm)
        for k, w in self.weights.items():
            so.adamw(w, self.grads[k], *self.moments[k], self.t, lr, weight_decay=0.0)
            self.grads[k].zero_()
        return norm


def make_batch(vocab: int, pairs: int, longest: int, seed: int):
    """Pairs of answers to the same prompt: the chosen one goes on by one fixed random function, the other at random."""
    g = torch.Generator().manual_seed(seed)
    follow = torch.randint(0, vocab, (vocab,), generator=torch.Generator().manual_seed(99))
    ids, targets, lengths = [], [], []
    for _ in range(pairs):
        prompt = torch.randint(0, vocab, (int(torch.randint(1, 8, (), generator=g)),), generator=g)
        for chosen in (True, False):
            n = int(torch.randint(2, longest, (), generator=g))
            answer = torch.randint(0, vocab, (n,), generator=g)
            if chosen:
                answer[0] = follow[prompt[-1]]
                for i in range(1, n):
                    answer[i] = follow[answer[i - 1]]
            tokens = torch.cat((prompt, answer))
            after = torch.cat((tokens[1:], torch.tensor([IGNORE])))
            after[:len(prompt) - 1] = IGNORE
            ids.append(tokens)
            targets.append(after)
            lengths.append(len(tokens))
    offsets = torch.cat((torch.zeros(1, dtype=torch.int64), torch.cumsum(torch.tensor(lengths), 0)))
    return Batch(torch.cat(ids).cuda(), torch.cat(targets).cuda(), offsets.cuda())


def train(steps: int = 40, vocab: int = 500, dim: int = 128, pairs: int = 32, longest: int = 24, lr: float = 0.01):
    """(loss, gradient norm) of each step."""
    model, start, seen = Model(vocab, dim), Model(vocab, dim), []
    for t in range(steps):
        batch = make_batch(vocab, pairs, longest, seed=t)
        batch.ref_logp, _ = start.forward(batch)
        loss, _ = model.preference(batch)
        seen.append(torch.stack((loss, model.step(lr))))
    so.check_device()
    return torch.stack(seen).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args()
    for t, (loss, norm) in enumerate(train(a.steps)):
        if t % max(1, a.steps // 10) == 0 or t == a.steps - 1:
            print("step %3d  loss %.4f  gradient norm %.3f" % (t, loss, norm))
