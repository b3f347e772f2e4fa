"""The stage-end operators written out in float64 on the CPU (test infrastructure;
shares no code with the library)."""
import torch

GROUP, FP8_MAX, TINY = 128, 448.0, 2.0 ** -126


def embed_grad(ids, dy, vocab, scale, padding=None):
    """(sum, sum of magnitudes, tokens per row)."""
    ids, d = ids.reshape(-1).long(), dy.reshape(-1, dy.shape[-1]).double()
    keep = (ids >= 0) & (ids < vocab)
    if padding is not None:
        keep &= ids != padding
    ids, d = ids[keep], d[keep]
    out, mag = (torch.zeros(vocab, d.shape[1], dtype=torch.float64) for _ in range(2))
    out.index_add_(0, ids, d)
    mag.index_add_(0, ids, d.abs())
    return out * scale, mag * abs(scale), torch.bincount(ids, minlength=vocab)


def groups(s):
    rows, dim = s.shape
    n = -(-dim // GROUP)
    return torch.nn.functional.pad(s, (0, n * GROUP - dim)).view(rows, n, GROUP)


def checkpoint32(s):
    """(q, scale) in fp32, operation by operation as the definition states them (bit-exact)."""
    g = groups(s.float())
    amax = g.abs().amax(-1)
    amax = torch.where(g.isnan().any(-1), torch.full_like(amax, float("inf")), amax)
    scale = (amax / FP8_MAX).clamp_min(TINY)
    q = (g * (1.0 / scale)[:, :, None]).reshape(s.shape[0], -1)[:, :s.shape[1]].to(torch.float8_e4m3fn)
    return q, scale


def dequantise(q, scale):
    return (groups(q.double()) * scale.double()[:, :, None]).reshape(q.shape[0], -1)[:, :q.shape[1]]


def norm_forward(s, gamma, eps):
    s = s.double()
    rstd = 1 / torch.sqrt((s * s).mean(-1) + eps)
    return s * rstd[:, None] * gamma.double(), rstd


def norm_backward(dy, ds, q, scale, rstd, gamma):
    """(dx, magnitude of dx's terms, dgamma, magnitude of its terms, y)."""
    n = dequantise(q, scale) * rstd.double()[:, None]
    dy, gamma, r = dy.double(), gamma.double(), rstd.double()[:, None]
    dn = dy * gamma
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    mag = r * (dn.abs() + n.abs() * (dn * n).abs().mean(-1, keepdim=True))
    if ds is not None:
        dx, mag = dx + ds.double(), mag + ds.double().abs()
    return dx, mag, (dy * n).sum(0), (dy * n).abs().sum(0), n * gamma


def head(h, w, target, ignore=-100, mean=True, grad_scale=1.0):
    h, w, target = h.double(), w.double(), target.long()
    valid = (target != ignore) & (target >= 0) & (target < w.shape[0])
    column = torch.where(valid, target, 0)
    logits = h @ w.T
    lse = torch.logsumexp(logits, 1)
    # the target's entries without the cancellation that even 64 bits meet where the loss is below 1e-16
    lt = logits.gather(1, column[:, None])
    others = torch.exp(torch.logsumexp(logits.scatter(1, column[:, None], -float("inf")), 1) - lt[:, 0])
    row = torch.where(valid, torch.where(others < 1e8, torch.log1p(others), lse - lt[:, 0]), torch.zeros_like(lse))
    count = int(valid.sum())
    f = (1.0 / max(count, 1) if mean else 1.0)
    d = torch.exp(logits - lse[:, None])
    d[torch.arange(len(target)), column] = torch.where(others.isinf(), torch.full_like(others, -1.0), -others / (1 + others))
    d = torch.where(valid[:, None], d, torch.zeros_like(d))
    g = f * grad_scale
    return {"loss": row.sum() * f, "row_loss": row, "lse": lse, "dh": d @ w * g, "dw": d.T @ h * g, "d": d,
            "factor": g, "loss_factor": f, "valid": valid, "logit_mag": (h.abs() @ w.abs().T).amax(1)}
