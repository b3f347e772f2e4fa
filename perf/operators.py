"""The measured cases of the pipeline's end stages: the embedding of the first stage and its gradient, the residual
RMSNorm with an 8-bit checkpoint and its backward pass, and the vocabulary head's cross entropy with its gradients.

Sizes come from the 1B layer (width 2048, vocabulary 128256, context 2048, batch 32) and the 7B-shaped layer (width
4096); the others are generic odd sizes.  `run` computes an operator in plain fp32 torch operations, or calls the
package's kernels when `own` is true.
"""
import math

import numpy as np
import torch

own = False

GROUP = 128       # values that share one scale of an 8-bit checkpoint
FP8_MAX = 448.0   # largest e4m3 value
TINY = 2.0 ** -126
IGNORE = -100     # target of a token that has no loss

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # the first stage's whole batch: 32 sequences of 2048 tokens looked up in the optimizer's fp32 weights
        {"name": "lookup_batch", "op": "embed_lookup", "tokens": 65536, "vocab": 128256, "dim": 2048,
         "table": "fp32", "out": "bf16", "scale": 1.0},
        # one short prompt, a bf16 table, the embedding scaled by sqrt(width); latency counts
        {"name": "lookup_prompt", "op": "embed_lookup", "tokens": 37, "vocab": 32001, "dim": 4096,
         "table": "bf16", "out": "bf16", "scale": 64.0},
        # the whole batch's embedding gradient as AdamW takes it: dense fp32 [vocab, width]
        {"name": "embgrad_batch", "op": "embed_grad", "tokens": 65536, "vocab": 128256, "dim": 2048,
         "dy": "bf16", "out": "fp32", "scale": 1.0},
        # a small micro-batch with odd sizes, the gradient kept in bf16
        {"name": "embgrad_small", "op": "embed_grad", "tokens": 777, "vocab": 32001, "dim": 1000,
         "dy": "bf16", "out": "bf16", "scale": 31.6},
        # the norm of one layer over the whole batch, its input kept in 8 bits for the backward pass
        {"name": "norm_batch", "op": "norm_forward", "rows": 65536, "dim": 2048, "type": "bf16", "residual": True},
        # a handful of tokens of the wide layer, nothing to add; latency counts
        {"name": "norm_few", "op": "norm_forward", "rows": 5, "dim": 4096, "type": "bf16", "residual": False},
        # the backward pass of the same batch from its checkpoint, with the recomputed norm output
        {"name": "normgrad_batch", "op": "norm_backward", "rows": 65536, "dim": 2048, "type": "bf16",
         "residual": True},
        # odd sizes in fp32, no gradient of the residual stream
        {"name": "normgrad_odd", "op": "norm_backward", "rows": 301, "dim": 1001, "type": "fp32", "residual": False},
        # evaluation loss of one 2048-token sequence
        {"name": "loss_eval", "op": "head_loss", "tokens": 2048, "vocab": 128256, "dim": 2048, "ignored": 0.0},
        # the loss of a single token over a smaller vocabulary; latency counts
        {"name": "loss_one", "op": "head_loss", "tokens": 1, "vocab": 32001, "dim": 4096, "ignored": 0.0},
        # the last stage's training step on a micro-batch of 4 sequences, a tenth of the tokens without a target
        {"name": "lossgrad_step", "op": "head_loss_grad", "tokens": 8192, "vocab": 128256, "dim": 2048,
         "ignored": 0.1},
        # a ragged fine-tuning batch: half of the tokens are prompts, no size a multiple of a tile
        {"name": "lossgrad_odd", "op": "head_loss_grad", "tokens": 333, "vocab": 50001, "dim": 1000, "ignored": 0.5},
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed_lookup", "embed_grad", "norm_forward", "norm_backward", "head_loss", "head_loss_grad"])
    if op in ("embed_lookup", "embed_grad"):
        vocab, dim = _between(rng, 1000, 128256), _between(rng, 64, 4096)
        tokens = min(_between(rng, 1, 65536), 65536 * 2048 // dim)
        vocab = min(vocab, 128256 * 2048 // dim)
        case = {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "scale": rng.choice([1.0, math.sqrt(dim)])}
        if op == "embed_lookup":
            return {**case, "table": rng.choice(["bf16", "fp32"]), "out": "bf16"}
        return {**case, "dy": "bf16", "out": rng.choice(["bf16", "fp32"])}
    if op in ("norm_forward", "norm_backward"):
        dim = _between(rng, 64, 8192)
        kind = rng.choice(["bf16", "bf16", "fp32"])
        rows = min(_between(rng, 1, 65536), 65536 * 2048 * 2 // (dim * BYTES[kind]))
        return {"op": op, "rows": rows, "dim": dim, "type": kind, "residual": rng.random() < 0.7}
    vocab, dim = _between(rng, 1000, 128256), _between(rng, 64, 4096)
    if rng.random() < 0.75:
        dim = (dim + 7) // 8 * 8  # most widths are multiples of 8
    tokens = max(1, min(_between(rng, 1, 8192), 8192 * 128256 * 2048 // (vocab * dim)))
    return {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "ignored": rng.choice([0.0, 0.1, 0.5])}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, kind, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(TYPES[kind])


def _token_ids(g, tokens, vocab):
    """Word frequencies fall off as 1 / rank: the rank is log-uniform, and ranks are spread over the vocabulary."""
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    return _spread(rank, vocab)


def _spread(rank, vocab):
    step = 40503
    while math.gcd(step, vocab) != 1:
        step += 2
    return rank * step % vocab


def _distinct(tokens, vocab):
    """Expected number of distinct ids among `tokens` of _token_ids."""
    k = np.arange(vocab, dtype=np.float64)
    p = np.log((k + 2) / (k + 1)) / math.log(vocab + 1)
    return float(np.sum(-np.expm1(tokens * np.log1p(-p))))


def _stream_rows(g, rows, dim, kind):
    """Rows of a residual stream: every row of its own size, a few channels far larger than the rest."""
    channel = torch.ones(dim, device="cuda")
    channel[torch.randint(0, dim, (max(1, dim // 256),), generator=g, device="cuda")] = 20.0
    size = torch.exp(torch.randn(rows, 1, generator=g, device="cuda") * 0.5)
    return (torch.randn(rows, dim, generator=g, device="cuda") * channel * size).to(TYPES[kind])


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "embed_lookup":
        return {**case, "ids": _token_ids(g, case["tokens"], case["vocab"]),
                "table": _normal(g, (case["vocab"], case["dim"]), case["table"], 0.02), "out": TYPES[case["out"]]}
    if op == "embed_grad":
        return {**case, "ids": _token_ids(g, case["tokens"], case["vocab"]),
                "dy": _normal(g, (case["tokens"], case["dim"]), case["dy"], 1e-3), "out": TYPES[case["out"]]}
    if op in ("norm_forward", "norm_backward"):
        rows, dim, kind = case["rows"], case["dim"], case["type"]
        s = {**case, "eps": 1e-5, "gamma": (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(TYPES[kind])}
        x = _stream_rows(g, rows, dim, kind)
        if op == "norm_forward":
            return {**s, "x": x, "r": _normal(g, (rows, dim), kind, 0.3) if case["residual"] else None}
        # what the forward pass kept, in the form in which it keeps it
        q, scale, rstd = _checkpoint(x.float(), s["eps"])
        return {**s, "q": q, "scales": scale, "rstd": rstd, "dy": _normal(g, (rows, dim), kind, 1e-3),
                "ds": _normal(g, (rows, dim), kind, 1e-3) if case["residual"] else None}
    tokens, vocab, dim = case["tokens"], case["vocab"], case["dim"]
    target = _token_ids(g, tokens, vocab)
    w = _normal(g, (vocab, dim), "bf16", 0.02)
    # a trained model's hidden states lean towards their target's row, some more than others
    lean = 10.0 * torch.rand(tokens, 1, generator=g, device="cuda") / (dim * 0.02 ** 2)
    h = (torch.randn(tokens, dim, generator=g, device="cuda") + lean * w[target].float()).to(torch.bfloat16)
    if case["ignored"]:
        out = torch.rand(tokens, generator=g, device="cuda") < case["ignored"]
        out[0] = False  # a batch without any target is not worth a step
        target[out] = IGNORE
    return {**case, "h": h, "w": w, "target": target}


# ---------------------------------------------------------------- plain forms

def _groups(s):
    rows, dim = s.shape
    n = -(-dim // GROUP)
    return torch.nn.functional.pad(s, (0, n * GROUP - dim)).view(rows, n, GROUP)


def _dequantised(q, scale, dim):
    return (_groups(q.float()) * scale[:, :, None]).view(q.shape[0], -1)[:, :dim]


def _checkpoint(s, eps):
    """8-bit values, their groups' scales and the reciprocal root mean square of fp32 rows."""
    g = _groups(s)
    scale = (g.abs().amax(-1) / FP8_MAX).clamp_min(TINY)
    q = (g * (1.0 / scale)[:, :, None]).view(s.shape[0], -1)[:, :s.shape[1]].contiguous().to(torch.float8_e4m3fn)
    return q, scale, torch.rsqrt(s.square().mean(-1) + eps)


def _plain_norm_forward(x, r, gamma, eps):
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    q, scale, rstd = _checkpoint(s.float(), eps)
    y = (s.float() * rstd[:, None] * gamma.float()).to(x.dtype)
    return {"s": s, "y": y, "q": q, "scale": scale, "rstd": rstd}


def _plain_norm_backward(dy, ds, q, scale, rstd, gamma):
    n = _dequantised(q, scale, dy.shape[1]) * rstd[:, None]
    dn = dy.float() * gamma.float()
    dx = rstd[:, None] * (dn - n * (dn * n).mean(-1, keepdim=True))
    if ds is not None:
        dx = dx + ds.float()
    return {"dx": dx.to(dy.dtype), "dgamma": (dy.float() * n).sum(0), "y": (n * gamma.float()).to(dy.dtype)}


def _plain_head(h, w, target, grad):
    hf, wf = h.float(), w.float()
    valid = target != IGNORE
    column = torch.where(valid, target, 0)[:, None]
    logits = hf @ wf.T
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    row_loss = torch.where(valid, (top + torch.log(total) - logits.gather(1, column))[:, 0], 0.0)
    count = valid.sum().clamp_min(1)
    out = {"loss": row_loss.sum() / count, "row_loss": row_loss}
    if grad:
        del logits
        p = e / total
        p.scatter_add_(1, column, torch.full_like(top, -1.0))
        p *= (valid / count)[:, None]
        out["dh"] = (p @ wf).to(h.dtype)
        out["dw"] = (p.T @ hf).to(w.dtype)
    return out


def _plain(s):
    op = s["op"]
    if op == "embed_lookup":
        return (s["table"][s["ids"]].float() * s["scale"]).to(s["out"])
    if op == "embed_grad":
        full = torch.zeros(s["vocab"], s["dim"], device="cuda")
        return full.index_add_(0, s["ids"], s["dy"].float() * s["scale"]).to(s["out"])
    if op == "norm_forward":
        return _plain_norm_forward(s["x"], s["r"], s["gamma"], s["eps"])
    if op == "norm_backward":
        return _plain_norm_backward(s["dy"], s["ds"], s["q"], s["scales"], s["rstd"], s["gamma"])
    return _plain_head(s["h"], s["w"], s["target"], op == "head_loss_grad")


# ---------------------------------------------------------------- the package's operators

def _own(s):
    from spectral_corrected_optimizer_gb300 import stage_ends as se
    op = s["op"]
    if op == "embed_lookup":
        return se.embed_lookup(s["table"], s["ids"], scale=s["scale"], dtype=s["out"])
    if op == "embed_grad":
        return se.embed_grad(s["ids"], s["dy"], s["vocab"], scale=s["scale"], dtype=s["out"])
    if op == "norm_forward":
        kept, x, y = se.residual_norm(s["x"], s["r"], s["gamma"], s["eps"])
        return {"s": x, "y": y, "q": kept.q, "scale": kept.scale, "rstd": kept.rstd}
    if op == "norm_backward":
        kept = se.NormCheckpoint(s["q"], s["scales"], s["rstd"])
        dx, dgamma, y = se.residual_norm_backward(s["dy"], kept, s["gamma"], ds=s["ds"], recompute=True)
        return {"dx": dx, "dgamma": dgamma, "y": y}
    if op == "head_loss":
        loss, row_loss = se.head_loss(s["h"], s["w"], s["target"], ignore_index=IGNORE)
        return {"loss": loss, "row_loss": row_loss}
    loss, row_loss, dh, dw = se.head_loss_grad(s["h"], s["w"], s["target"], ignore_index=IGNORE, dtype=torch.bfloat16)
    return {"loss": loss, "row_loss": row_loss, "dh": dh, "dw": dw}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op == "embed_lookup":
        n, d = case["tokens"], case["dim"]
        rows = _distinct(n, case["vocab"])
        return {"bytes": 8 * n + rows * d * BYTES[case["table"]] + n * d * BYTES[case["out"]], "flops": n * d}
    if op == "embed_grad":
        n, d = case["tokens"], case["dim"]
        return {"bytes": 8 * n + n * d * BYTES[case["dy"]] + case["vocab"] * d * BYTES[case["out"]], "flops": 2 * n * d}
    if op in ("norm_forward", "norm_backward"):
        n, d, b = case["rows"], case["dim"], BYTES[case["type"]]
        kept = n * d + 4 * n * -(-d // GROUP) + 4 * n
        tensors = (4 if case["residual"] else 2) if op == "norm_forward" else (4 if case["residual"] else 3)
        return {"bytes": kept + tensors * n * d * b + d * b + (4 * d if op == "norm_backward" else 0),
                "flops": 8 * n * d}
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    kept = n * (1 - case["ignored"])
    grad = op == "head_loss_grad"
    return {"bytes": (n * d * 2 + v * d * 2) * (2 if grad else 1) + 12 * n, "flops": 2 * kept * v * d * (3 if grad else 1)}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_embed_grad(s):
    """Sums over the tokens of each id, by a sort of the ids and differences of running sums within blocks of columns."""
    order = torch.argsort(s["ids"], stable=True)
    ids, counts = torch.unique_consecutive(s["ids"][order], return_counts=True)
    ends = torch.cumsum(counts, 0) - 1
    full = torch.zeros(s["vocab"], s["dim"], device="cuda", dtype=torch.float64)
    for c in range(0, s["dim"], 256):
        run_sum = torch.cumsum(s["dy"][order, c:c + 256].double(), 0)[ends]
        full[ids, c:c + 256] = torch.diff(run_sum, dim=0, prepend=torch.zeros_like(run_sum[:1])) * s["scale"]
    return full


def _exact_values8(s, scale, dim):
    """e4m3 neighbours of s / scale by the format's spacing: 3 bits below the leading one, 2^-9 at the least."""
    v = (_groups(s) / scale[:, :, None]).view(s.shape[0], -1)[:, :dim]
    spacing = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / spacing) * spacing


def _exact_head(s, grad):
    h, w, target = s["h"].double(), s["w"].double(), s["target"]
    n = h.shape[0]
    count = max(1, int((target != IGNORE).sum()))
    row_loss = torch.zeros(n, device="cuda", dtype=torch.float64)
    dh = torch.zeros_like(h) if grad else None
    dw = torch.zeros_like(w) if grad else None
    for rows in torch.nonzero(target != IGNORE)[:, 0].split(1024):
        logits = torch.einsum("nd,vd->nv", h[rows], w)
        lse = torch.logsumexp(logits, 1)
        row_loss[rows] = lse - logits[torch.arange(len(rows), device="cuda"), target[rows]]
        if grad:
            d = torch.exp(logits - lse[:, None])
            del logits
            d[torch.arange(len(rows), device="cuda"), target[rows]] -= 1
            d /= count
            dh[rows] = d @ w
            dw.addmm_(d.T, h[rows])
    out = {"loss": row_loss.sum() / count, "row_loss": row_loss}
    return {**out, "dh": dh, "dw": dw} if grad else out


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "embed_lookup":
        return torch.index_select(s["table"], 0, s["ids"]).double() * s["scale"]
    if op == "embed_grad":
        return _exact_embed_grad(s)
    if op == "norm_forward":
        x = s["x"].double()
        if s["r"] is not None:
            x = (x + s["r"].double()).to(s["x"].dtype).double()  # the stream is held in its own type
        gamma, dim = s["gamma"].double(), case["dim"]
        scale = (_groups(x).abs().amax(-1) / 448).clamp_min(2.0 ** -126)
        rstd = 1 / torch.sqrt((x * x).sum(-1) / dim + s["eps"])
        return {"s": x, "y": x * rstd[:, None] * gamma, "q": _exact_values8(x, scale, dim), "scale": scale, "rstd": rstd}
    if op == "norm_backward":
        dim = case["dim"]
        dy, gamma, rstd = s["dy"].double(), s["gamma"].double(), s["rstd"].double()[:, None]
        x = (_groups(s["q"].double()) * s["scales"].double()[:, :, None]).flatten(1)[:, :dim]
        y = x * rstd * gamma
        mean = (dy * y).sum(-1, keepdim=True) / dim
        dx = rstd * gamma * dy - rstd ** 2 * x * mean
        if s["ds"] is not None:
            dx = dx + s["ds"].double()
        return {"dx": dx, "dgamma": torch.einsum("nd,nd->d", dy, x * rstd), "y": y}
    return _exact_head(s, op == "head_loss_grad")
