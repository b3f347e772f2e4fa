"""The fine-tuning operators written out in float64 on the CPU (test infrastructure;
shares no code with the library)."""
import math

import torch


def norm_forward(s, gamma, beta, eps):
    """(y, mean, rstd) of the rows of s."""
    s, gamma = s.double(), gamma.double()
    mean = s.mean(-1)
    d = s - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(-1) + eps)
    y = d * rstd[:, None] * gamma
    return (y if beta is None else y + beta.double()), mean, rstd


def norm_backward(dy, ds, s, mean, rstd, gamma):
    """(dx, magnitude of dx's terms, dgamma, its terms', dbeta, its terms')."""
    dy, r = dy.double(), rstd.double()[:, None]
    n = (s.double() - mean.double()[:, None]) * r
    g = dy * gamma.double()
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    mag = r * (g.abs() + g.abs().mean(-1, keepdim=True) + n.abs() * (g * n).abs().mean(-1, keepdim=True))
    if ds is not None:
        dx, mag = dx + ds.double(), mag + ds.double().abs()
    return dx, mag, (dy * n).sum(0), (dy * n).abs().sum(0), dy.sum(0), dy.abs().sum(0)


def spans(offsets):
    o = [int(x) for x in offsets]
    return [slice(a, b) for a, b in zip(o[:-1], o[1:])]


def counting(offsets, tokens, mask):
    """The tokens that lie in a sequence and count."""
    on = torch.zeros(tokens, dtype=torch.bool)
    for s in spans(offsets):
        on[s] = True
    return on if mask is None else on & mask.bool()


def preference(logp, ref, offsets, beta, kind, smoothing=0.0, average=False, mask=None, mean=True, grad_scale=1.0):
    """Values and the magnitudes that their errors are measured by."""
    on = counting(offsets, len(logp), mask)
    d = logp.double() if ref is None else logp.double() - ref.double()
    d = torch.where(on, d, torch.zeros_like(d))
    all_spans = spans(offsets)
    number = torch.tensor([int(on[s].sum()) for s in all_spans]).double().clamp_min(1)
    share = 1 / number if average else torch.ones_like(number)
    rewards = beta * share * torch.stack([d[s].sum() for s in all_spans]) if all_spans else torch.zeros(0).double()
    size = beta * share * torch.stack([d[s].abs().sum() for s in all_spans]) if all_spans else torch.zeros(0).double()
    rewards, size = rewards.view(-1, 2), size.view(-1, 2)
    delta = rewards[:, 0] - rewards[:, 1]
    if kind == "logistic":
        up, down = torch.sigmoid(delta), torch.sigmoid(-delta)
        loss = -torch.nn.functional.logsigmoid(delta) * (1 - smoothing)
        if smoothing:
            loss = loss - torch.nn.functional.logsigmoid(-delta) * smoothing
        slope, slope_mag = smoothing * up - (1 - smoothing) * down, smoothing * up + (1 - smoothing) * down
    elif kind == "hinge":
        loss = (1 - delta).clamp_min(0)
        slope = -(delta < 1).double()
        slope_mag = slope.abs()
    else:
        gap = delta / beta - 1 / (2 * beta)
        loss, slope = gap ** 2, 2 * gap / beta
        slope_mag = slope.abs()
    pairs = len(delta)
    f = 1 / max(pairs, 1) if mean else 1.0
    dlogp = torch.zeros_like(d)
    factor = torch.zeros_like(d)
    for i, s in enumerate(all_spans):
        factor[s] = (beta * share[i] * f * grad_scale) * (1 if i % 2 == 0 else -1)
        dlogp[s] = slope[i // 2] * factor[s]
    zero = torch.zeros_like(d)
    return {"loss": loss.sum() * f, "pair_loss": loss, "rewards": rewards, "size": size, "delta": delta, "slope": slope,
            "slope_mag": slope_mag, "dlogp": torch.where(on, dlogp, zero), "factor": torch.where(on, factor, zero), "on": on,
            "f": f}


def policy(logp, old, advantages, offsets, ref=None, mask=None, low=0.2, high=0.2, kl_coef=0.0, reduction="token",
           grad_scale=1.0, per_sequence=False):
    tokens = len(logp)
    count = len(offsets) - 1
    on = counting(offsets, tokens, mask)
    lp = torch.where(on, logp.double(), torch.zeros(tokens).double())
    lo = torch.where(on, old.double(), torch.zeros(tokens).double())
    a = advantages.double()
    if per_sequence:
        a = torch.zeros(tokens).double()
        for i, s in enumerate(spans(offsets)):
            a[s] = advantages[i].double()
    a = torch.where(on, a, torch.zeros_like(a))
    d = lp - lo
    ratio = torch.exp(d)
    clipped = torch.where(a >= 0, d > math.log(1 + high), d < (math.log(1 - low) if low < 1 else -math.inf))
    bounded = torch.where(clipped, torch.where(a >= 0, 1.0 + high, 1.0 - low).double(), ratio)
    gain = a * bounded
    slope = torch.where(clipped, torch.zeros_like(a), -a * ratio)
    kl, q, e = torch.zeros_like(a), torch.zeros_like(a), torch.zeros_like(a)
    if ref is not None:
        q = torch.where(on, ref.double(), torch.zeros_like(a)) - lp
        e = torch.expm1(q)
        kl = torch.where(q.abs() < 1e-3, q * q * (0.5 + q / 6 + q * q / 24), e - q)
        slope = slope - kl_coef * e
    weight = torch.zeros(tokens).double()
    if reduction == "token":
        weight[on] = 1 / max(int(on.sum()), 1)
    elif reduction == "sum":
        weight[on] = 1.0
    else:
        for s in spans(offsets):
            weight[s] = on[s].double() / max(int(on[s].sum()), 1) / count
    parts = torch.stack([(weight * torch.where(on, t, torch.zeros_like(a))).sum() for t in (-gain, kl, clipped.double())])
    return {"loss": parts[0] + kl_coef * parts[1], "parts": parts, "dlogp": slope * weight * grad_scale, "on": on, "d": d, "q": q,
            "e": e, "gain": gain.abs() * on, "kl": kl * on, "slope": slope, "weight": weight, "clipped": clipped & on,
            "ratio": ratio}


def norm_of(tensors, scale=1.0, norm_type=2.0):
    values = [t.double().flatten() * abs(scale) for t in tensors if t.numel()]
    if not values:
        return 0.0
    if norm_type == math.inf:
        return float(torch.stack([v.abs().max() for v in values]).max())
    return float(torch.sqrt(sum((v * v).sum() for v in values)))
