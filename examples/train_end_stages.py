"""Trains the two end stages of a pipeline on one GPU, with the masked boundary between them.

    python examples/train_end_stages.py [--steps 60]

A toy language -- the next token is a fixed function of the current one -- is learned by the smallest model that has
every operator of the end stages and of the boundary:

  stage 0   x = embed_lookup(E, ids), sent as mask_pack(x): K of the H values of each token (key design 1 of
            "Communication-Efficient LLM Adaptation over Decentralized GPU Meshes")
  stage 1   h = mask_unpack(...), s = h + (h of the token before), y = RMSNorm(s) * gamma, with s kept in 8 bits;
            loss = cross entropy of y against W over the vocabulary

The backward pass mirrors it: head_loss_grad gives dL/dy and adds dL/dW, residual_norm_backward works from the 8-bit
checkpoint, the boundary's gradient travels masked with the same indices, embed_grad adds up dL/dE.  Gradients of the
micro-batches accumulate in fp32 and the framework's AdamW steps the fp32 weights.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import spectral_corrected_optimizer_gb300 as so  # noqa: E402
from spectral_corrected_optimizer_gb300 import stage_ends as se  # noqa: E402

IGNORE = -100


class EndStages:
    """Weights, gradients and AdamW state of both stages."""

    def __init__(self, vocab: int, dim: int, p: float = 0.5, seed: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.vocab, self.dim, self.K = vocab, dim, so.mask_keep_count(p, dim)
        self.weights = {"embed": torch.randn(vocab, dim, generator=g, device="cuda"),
                        "gamma": torch.ones(dim, device="cuda"),
                        "head": torch.randn(vocab, dim, generator=g, device="cuda") * dim ** -0.5}
        self.grads = {k: torch.zeros_like(w) for k, w in self.weights.items()}
        self.moments = {k: (torch.zeros_like(w), torch.zeros_like(w)) for k, w in self.weights.items()}
        self.t = 0

    def micro_batch(self, ids, targets, step: int, batch_id: int, grad_scale: float):
        """Loss of one micro-batch; its gradients are added to self.grads."""
        rows = ids.numel()
        gamma, head = self.weights["gamma"].bfloat16(), self.weights["head"].bfloat16()
        # stage 0, forward
        x = se.embed_lookup(self.weights["embed"], ids, dtype=torch.bfloat16)
        sent = so.mask_pack(x, self.K, 0, step, batch_id)
        # stage 1, forward and backward
        h = so.mask_unpack(sent, self.dim, 0, step, batch_id)
        before = torch.cat((torch.zeros_like(h[:1]), h[:-1]))
        kept, s, y = se.residual_norm(h, before, gamma)
        loss, _, dy, _ = se.head_loss_grad(y, head, targets, ignore_index=IGNORE, grad_scale=grad_scale,
                                           dw=self.grads["head"], accumulate=True)
        ds, dgamma, _ = se.residual_norm_backward(dy, kept, gamma)
        self.grads["gamma"] += dgamma
        dh = ds + torch.cat((ds[1:], torch.zeros_like(ds[:1])))
        back = so.mask_pack(dh, self.K, 0, step, batch_id)
        # stage 0, backward
        dx = so.mask_unpack(back, self.dim, 0, step, batch_id)
        se.embed_grad(ids, dx, self.vocab, out=self.grads["embed"], accumulate=True)
        assert rows == dx.shape[0]
        return loss

    def step(self, lr: float):
        self.t += 1
        for k, w in self.weights.items():
            so.adamw(w, self.grads[k], *self.moments[k], self.t, lr)
            self.grads[k].zero_()


def batches(vocab: int, tokens: int, count: int, seed: int):
    """Token ids and their successors under a fixed random function; the last token of a batch has no target."""
    g = torch.Generator().manual_seed(seed)
    successor = torch.randint(0, vocab, (vocab,), generator=g)
    for _ in range(count):
        ids = torch.randint(0, vocab, (tokens,), generator=g)
        targets = successor[ids]
        targets[-1] = IGNORE
        yield ids.cuda(), targets.cuda()


def train(steps: int = 60, vocab: int = 1000, dim: int = 256, tokens: int = 2048, micro: int = 2, lr: float = 0.02):
    """The mean loss of each step."""
    model, losses = EndStages(vocab, dim), []
    data = batches(vocab, tokens, steps * micro, seed=1)
    for t in range(steps):
        parts = [model.micro_batch(*next(data), step=t, batch_id=m, grad_scale=1.0 / micro) for m in range(micro)]
        model.step(lr)
        losses.append(sum(parts) / micro)
    so.check_device()
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    a = ap.parse_args()
    got = train(a.steps)
    for t in range(0, len(got), max(1, len(got) // 10)):
        print("step %3d  loss %.4f" % (t, got[t]))
    print("step %3d  loss %.4f" % (len(got) - 1, got[-1]))
