"""The measured cases of the fine-tuning step: LayerNorm with its gradients, the vocabulary head's gradient for losses over
log-probabilities, the preference and the clipped policy loss, and the global gradient norm with clipping.

Sizes come from the 1B layer (width 2048, vocabulary 128256, context 2048, batch 32) and the 7B-shaped layer (width
4096); the others are generic odd sizes.  `run` computes an operator in plain fp32 torch operations, or calls the
package's kernels when `own` is true.
"""
import math

import torch

own = False

IGNORE = -100     # target of a token that has no log-probability
EPS = 1e-5
LOG2E = math.log2(math.e)

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


def listed():
    return [
        # the norm of one layer over the whole batch of 32 sequences of 2048 tokens, residual sum included
        {"name": "norm_batch", "op": "norm_forward", "rows": 65536, "dim": 2048, "type": "bf16", "residual": True,
         "bias": True},
        # a handful of tokens of the wide layer, nothing to add; latency counts
        {"name": "norm_few", "op": "norm_forward", "rows": 5, "dim": 4096, "type": "bf16", "residual": False,
         "bias": True},
        # the backward pass of the same batch, the residual stream's gradient added
        {"name": "normgrad_batch", "op": "norm_backward", "rows": 65536, "dim": 2048, "type": "bf16",
         "residual": True, "bias": True},
        # odd sizes in fp32, a norm without a bias, no gradient of the residual stream
        {"name": "normgrad_odd", "op": "norm_backward", "rows": 301, "dim": 1001, "type": "fp32", "residual": False,
         "bias": False},
        # the head's gradient for one pair of 2048-token sequences, half of whose tokens are the prompt
        {"name": "headgrad_pair", "op": "head_backward", "tokens": 4096, "vocab": 128256, "dim": 2048,
         "ignored": 0.5, "still": 0.0},
        # a ragged rollout batch: prompts left out, a tenth of the answers clipped, no size a multiple of a tile
        {"name": "headgrad_odd", "op": "head_backward", "tokens": 333, "vocab": 50001, "dim": 1000, "ignored": 0.3,
         "still": 0.1},
        # all pairs of an optimizer step: 1024 pairs of sequences of 2048 tokens on average, prompts masked
        {"name": "pairs_step", "op": "preference", "pairs": 1024, "length": 2048, "kind": "logistic",
         "smoothing": 0.1, "average": False, "mask": True, "reference": True, "pad": 0},
        # one pair of short answers; latency counts
        {"name": "pairs_one", "op": "preference", "pairs": 1, "length": 45, "kind": "square", "smoothing": 0.0,
         "average": True, "mask": False, "reference": True, "pad": 6},
        # the rollouts of an optimizer step, 2048 answers of 2048 tokens on average, one advantage per answer
        {"name": "rollouts_step", "op": "policy", "sequences": 2048, "length": 2048, "per_token": False,
         "reference": True, "mask": True, "reduction": "token", "pad": 0},
        # a micro-batch of 7 answers, an advantage per token, every answer with the same weight
        {"name": "rollouts_micro", "op": "policy", "sequences": 7, "length": 331, "per_token": True,
         "reference": False, "mask": True, "reduction": "sequence", "pad": 11},
        # all gradients of the 1B model, 16 layers of 9 tensors, the embedding and the last norm, clipped in fp32
        {"name": "clip_model", "op": "clip", "layers": 16, "tensors": 0, "values": 0, "type": "fp32", "out": "fp32",
         "scale": 1.0, "clipped": 0.5, "limit": 2.0},
        # one layer's bf16 gradients clipped into the fp32 ones that AdamW takes
        {"name": "clip_layer", "op": "clip", "layers": 1, "tensors": 0, "values": 0, "type": "bf16", "out": "fp32",
         "scale": 0.25, "clipped": 0.3, "limit": 2.0},
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_forward", "norm_backward", "head_backward", "preference", "policy", "grad_norm", "clip"])
    if op in ("norm_forward", "norm_backward"):
        dim = _between(rng, 64, 8192)
        if rng.random() < 0.6:
            dim = (dim + 7) // 8 * 8  # most widths are multiples of 8
        kind = rng.choice(["bf16", "bf16", "fp32"])
        rows = min(_between(rng, 1, 65536), 65536 * 2048 * 2 // (dim * BYTES[kind]))
        return {"op": op, "rows": rows, "dim": dim, "type": kind, "residual": rng.random() < 0.6,
                "bias": rng.random() < 0.8}
    if op == "head_backward":
        vocab, dim = _between(rng, 1000, 128256), _between(rng, 64, 4096)
        if rng.random() < 0.75:
            dim = (dim + 7) // 8 * 8
        tokens = max(1, min(_between(rng, 1, 4096), 4096 * 128256 * 2048 // (vocab * dim)))
        return {"op": op, "tokens": tokens, "vocab": vocab, "dim": dim, "ignored": rng.choice([0.5, 0.7, 0.9]),
                "still": rng.choice([0.0, 0.1])}
    if op == "preference":
        pairs = _between(rng, 1, 2048)
        length = min(_between(rng, 4, 8192), 2 * 1024 * 2048 // (2 * pairs) + 1)
        kind = rng.choice(["logistic", "logistic", "hinge", "square"])
        return {"op": op, "pairs": pairs, "length": length, "kind": kind,
                "smoothing": rng.choice([0.0, 0.1]) if kind == "logistic" else 0.0, "average": rng.random() < 0.3,
                "mask": rng.random() < 0.7, "reference": rng.random() < 0.8, "pad": rng.choice([0, 0, 5, 1000])}
    if op == "policy":
        sequences = _between(rng, 1, 4096)
        length = min(_between(rng, 4, 16384), 2048 * 2048 // sequences + 1)
        return {"op": op, "sequences": sequences, "length": length, "per_token": rng.random() < 0.5,
                "reference": rng.random() < 0.6, "mask": rng.random() < 0.7,
                "reduction": rng.choice(["token", "sequence"]), "pad": rng.choice([0, 0, 5, 1000])}
    tensors, kind = _between(rng, 1, 60), rng.choice(["bf16", "fp32"])
    case = {"op": op, "layers": 0, "tensors": tensors, "values": tensors + _between(rng, 1000, 60_000_000),
            "type": kind, "limit": rng.choice([2.0, 2.0, 2.0, math.inf])}
    if op == "grad_norm":
        return case
    return {**case, "out": rng.choice([kind, "fp32"]), "scale": rng.choice([1.0, 0.125]),
            "clipped": rng.choice([0.1, 0.9, 3.0])}


# ---------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, kind, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(TYPES[kind])


def _stream_rows(g, rows, dim, kind):
    """Rows of a residual stream: every row of its own size and with a mean, a few channels far larger than the rest."""
    channel = torch.ones(dim, device="cuda")
    channel[torch.randint(0, dim, (max(1, dim // 256),), generator=g, device="cuda")] = 20.0
    size = torch.exp(torch.randn(rows, 1, generator=g, device="cuda") * 0.5)
    middle = 0.5 * torch.randn(rows, 1, generator=g, device="cuda")
    return ((torch.randn(rows, dim, generator=g, device="cuda") * channel + middle) * size).to(TYPES[kind])


def _token_ids(g, tokens, vocab):
    """Word frequencies fall off as 1 / rank: the rank is log-uniform, and ranks are spread over the vocabulary."""
    u = torch.rand(tokens, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp_(0, vocab - 1)
    step = 40503
    while math.gcd(step, vocab) != 1:
        step += 2
    return rank * step % vocab


def _head_state(h, w, target):
    """What the forward pass keeps of each token: a whole number m, 1 / sum_v 2^(log2(e) l_v - m), and one minus the
    target's probability."""
    kept = torch.zeros(3, len(target), device="cuda")
    wf = w.float()
    for rows in torch.nonzero(target != IGNORE)[:, 0].split(1024):
        l2 = (h[rows].float() @ wf.T).double() * LOG2E
        m = l2.amax(1).ceil()
        e = torch.exp2(l2 - m[:, None])
        del l2
        total = e.sum(1)
        e.scatter_(1, target[rows][:, None], 0.0)
        kept[0, rows], kept[1, rows], kept[2, rows] = m.float(), (1 / total).float(), (e.sum(1) / total).float()
    return kept


def _lengths(count, length):
    """Many short sequences and a few of three times the average; sum about count * length, whatever the seed."""
    q = (torch.arange(count, dtype=torch.float64) + 0.5) / count
    return torch.round(3 * length * q * q).long() if count > 2 else torch.full((count,), length)


def _offsets(g, count, length):
    lengths = _lengths(count, length).cuda()[torch.randperm(count, generator=g, device="cuda")]
    return torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(lengths, 0)))


def _answers(g, offsets, tokens):
    """True at the tokens of a sequence's answer: its prompt takes up to half of it."""
    count = len(offsets) - 1
    start = offsets[:-1] + ((offsets[1:] - offsets[:-1]) * 0.5 * torch.rand(count, generator=g, device="cuda")).long()
    at = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(offsets, at, right=True) - 1
    return (seq < count) & (at >= start[seq.clamp_max(count - 1)])


def _log_probabilities(g, tokens):
    """A trained model's: most tokens near certain, some far from it."""
    return -torch.empty(tokens, device="cuda").exponential_(1.0, generator=g).square_() * 0.5


def _sizes(case):
    """The sizes of the gradients, those that lie in one buffer together: a whole model's lie in one for each layer."""
    if case["layers"]:
        layer = [2048 * 2048, 512 * 2048, 512 * 2048, 2048 * 2048, 8192 * 2048, 8192 * 2048, 2048 * 8192, 2048, 2048]
        return [[n] for n in layer] if case["layers"] == 1 else [layer] * case["layers"] + [[128256 * 2048, 2048]]
    n = case["tensors"]
    weights = [1 / (1 + 7919 * i % n) ** 2 for i in range(n)]  # a few large tensors and many small ones, in any order
    return [[1 + int((case["values"] - n) * x / sum(weights))] for x in weights]


def _values(case):
    return sum(map(sum, _sizes(case)))


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op in ("norm_forward", "norm_backward"):
        rows, dim, kind = case["rows"], case["dim"], case["type"]
        s = {**case, "gamma": (1 + 0.2 * torch.randn(dim, generator=g, device="cuda")).to(TYPES[kind]),
             "beta": _normal(g, (dim,), kind, 0.1) if case["bias"] else None, "x": _stream_rows(g, rows, dim, kind)}
        if op == "norm_forward":
            return {**s, "r": _normal(g, (rows, dim), kind, 0.3) if case["residual"] else None}
        # what the forward pass kept of its rows
        x = s["x"].float()
        mean = x.mean(-1)
        rstd = torch.rsqrt((x - mean[:, None]).square().mean(-1) + EPS)
        return {**s, "mean": mean, "rstd": rstd, "dy": _normal(g, (rows, dim), kind, 1e-3),
                "ds": _normal(g, (rows, dim), kind, 1e-3) if case["residual"] else None}
    if op == "head_backward":
        tokens, vocab, dim = case["tokens"], case["vocab"], case["dim"]
        target = _token_ids(g, tokens, vocab)
        w = _normal(g, (vocab, dim), "bf16", 0.02)
        # a trained model's hidden states lean towards their target's row, some more than others
        lean = 10.0 * torch.rand(tokens, 1, generator=g, device="cuda") / (dim * 0.02 ** 2)
        h = (torch.randn(tokens, dim, generator=g, device="cuda") + lean * w[target].float()).to(torch.bfloat16)
        out = torch.rand(tokens, generator=g, device="cuda") < case["ignored"]
        out[0] = False  # a batch without any answer is not worth a step
        target[out] = IGNORE
        dlogp = torch.randn(tokens, generator=g, device="cuda") / tokens
        still = torch.rand(tokens, generator=g, device="cuda") < case["still"]
        still[0] = False
        dlogp[still] = 0.0
        return {**case, "h": h, "w": w, "target": target, "dlogp": dlogp, "kept": _head_state(h, w, target)}
    if op == "preference":
        offsets = _offsets(g, 2 * case["pairs"], case["length"])
        tokens = int(offsets[-1]) + case["pad"]
        logp = _log_probabilities(g, tokens)
        ref = logp + 0.1 * torch.randn(tokens, generator=g, device="cuda") if case["reference"] else None
        return {**case, "offsets": offsets, "logp": logp, "ref": ref, "beta": 0.1,
                "valid": _answers(g, offsets, tokens) if case["mask"] else None}
    if op == "policy":
        offsets = _offsets(g, case["sequences"], case["length"])
        tokens = int(offsets[-1]) + case["pad"]
        logp = _log_probabilities(g, tokens)
        old = logp + 0.15 * torch.randn(tokens, generator=g, device="cuda")
        ref = logp + 0.3 * torch.randn(tokens, generator=g, device="cuda") if case["reference"] else None
        advantage = torch.randn(tokens if case["per_token"] else case["sequences"], generator=g, device="cuda")
        return {**case, "offsets": offsets, "logp": logp, "old": old, "ref": ref, "advantage": advantage,
                "valid": _answers(g, offsets, tokens) if case["mask"] else None, "low": 0.2, "high": 0.28,
                "kl": 0.04 if case["reference"] else 0.0}
    buffers = _sizes(case)
    sizes = [n for b in buffers for n in b]
    # parameters' gradients differ in size by orders of magnitude
    stds = iter((1e-3 * torch.exp(1.5 * torch.randn(len(sizes), generator=g, device="cuda"))).tolist())
    grads = []
    for b in buffers:
        flat = _normal(g, (sum(b),), case["type"])
        grads += flat.split(b)
    for x in grads:
        x *= next(stds)
    s = {**case, "grads": grads}
    if op == "clip":
        # the limit: a share of the norm that these gradients have on average, at times above it
        typical = 1e-3 * math.sqrt(sum(n * math.exp(2.25) for n in sizes)) if case["limit"] == 2.0 else 0.1
        s["most"] = case["clipped"] * case["scale"] * typical
        s["flat"] = [torch.empty(sum(b), dtype=TYPES[case["out"]], device="cuda") for b in buffers]
        s["outs"] = [x for flat, b in zip(s["flat"], buffers) for x in flat.split(b)]
    return s


# ---------------------------------------------------------------- plain forms

def _plain_norm_forward(x, r, gamma, beta):
    s = x if r is None else (x.float() + r.float()).to(x.dtype)
    f = s.float()
    mean = f.mean(-1)
    d = f - mean[:, None]
    rstd = torch.rsqrt(d.square().mean(-1) + EPS)
    y = d * rstd[:, None] * gamma.float()
    if beta is not None:
        y = y + beta.float()
    return {"s": s, "y": y.to(x.dtype), "mean": mean, "rstd": rstd}


def _plain_norm_backward(dy, x, mean, rstd, gamma, ds, bias):
    n = (x.float() - mean[:, None]) * rstd[:, None]
    d = dy.float()
    g = d * gamma.float()
    dx = rstd[:, None] * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    if ds is not None:
        dx = dx + ds.float()
    out = {"dx": dx.to(dy.dtype), "dgamma": (d * n).sum(0)}
    return {**out, "dbeta": d.sum(0)} if bias else out


def _plain_head_backward(h, w, target, dlogp, kept):
    hf, wf = h.float(), w.float()
    m, inv, rest = kept[0, :, None], kept[1, :, None], kept[2, :, None]
    valid = (target != IGNORE) & (dlogp != 0)
    p = torch.exp2((hf @ wf.T) * LOG2E - m) * inv
    p.scatter_(1, torch.where(valid, target, 0)[:, None], -rest)  # softmax - onehot
    p *= torch.where(valid, -dlogp, 0.0)[:, None]
    p[~valid] = 0.0
    return {"dh": (p @ wf).to(h.dtype), "dw": (p.T @ hf).to(w.dtype)}


def _sequences(offsets, tokens, valid):
    """The sequence of each token, and whether it counts."""
    count = len(offsets) - 1
    seq = torch.searchsorted(offsets, torch.arange(tokens, device="cuda"), right=True) - 1
    counts = (seq >= 0) & (seq < count)
    return seq.clamp(0, count - 1), counts if valid is None else counts & valid


def _plain_preference(s):
    logp, offsets, beta, eps = s["logp"], s["offsets"], s["beta"], s["smoothing"]
    pairs = s["pairs"]
    seq, counts = _sequences(offsets, len(logp), s["valid"])
    d = logp.double() if s["ref"] is None else logp.double() - s["ref"].double()
    d = torch.where(counts, d, 0.0)
    total = torch.zeros(2 * pairs, dtype=torch.float64, device="cuda").index_add_(0, seq, d)
    share = torch.ones_like(total)
    if s["average"]:
        number = torch.zeros_like(total).index_add_(0, seq, counts.double())
        share = 1 / number.clamp_min(1)
    rewards = (beta * total * share).view(pairs, 2)
    delta = rewards[:, 0] - rewards[:, 1]
    if s["kind"] == "logistic":
        soft = torch.log1p(torch.exp(-delta.abs()))
        loss = (1 - eps) * (soft + (-delta).clamp_min(0)) + eps * (soft + delta.clamp_min(0))
        slope = 1 / (1 + torch.exp(-delta)) - (1 - eps)
    elif s["kind"] == "hinge":
        loss = (1 - delta).clamp_min(0)
        slope = -(delta < 1).double()
    else:
        gap = delta / beta - 1 / (2 * beta)
        loss, slope = gap * gap, 2 * gap / beta
    slope = torch.stack((slope, -slope), 1).view(-1) * beta * share / pairs
    return {"loss": loss.mean().float(), "pair_loss": loss.float(), "rewards": rewards.float(),
            "dlogp": torch.where(counts, slope[seq], 0.0).float()}


def _plain_policy(s):
    logp, offsets = s["logp"], s["offsets"]
    count = len(offsets) - 1
    seq, counts = _sequences(offsets, len(logp), s["valid"])
    a = s["advantage"] if s["per_token"] else s["advantage"][seq]
    far = logp.double() - s["old"].double()  # whether a token is clipped is decided in 64 bits
    ratio = torch.exp(far).float()
    clipped = torch.where(a >= 0, far > math.log1p(s["high"]), far < math.log1p(-s["low"]))
    edge = torch.where(a >= 0, 1 + s["high"], 1 - s["low"])
    gain = a * torch.where(clipped, edge, ratio)
    slope = torch.where(clipped, 0.0, -a * ratio)
    kl = torch.zeros_like(gain)
    if s["ref"] is not None:
        q = s["ref"] - logp
        e = torch.expm1(q)
        kl = e - q
        slope = slope - s["kl"] * e
    if s["reduction"] == "token":
        weight = (1 / counts.sum().clamp_min(1)).expand(len(logp))
    else:
        number = torch.zeros(count, device="cuda").index_add_(0, seq, counts.float())
        weight = (1 / (number.clamp_min(1) * count))[seq]
    weight = torch.where(counts, weight, 0.0).double()
    terms = torch.stack((-gain, kl, clipped.float())).double()
    part = torch.where(counts, terms, 0.0) @ weight
    return {"loss": (part[0] + s["kl"] * part[1]).float(), "parts": part.float(),
            "dlogp": torch.where(counts, slope * weight.float(), 0.0)}


def _plain_norm(grads, scale, limit):
    if limit == math.inf:
        return scale * torch.stack([x.abs().amax().float() for x in grads]).amax()
    squares = torch.stack([x.float().square().sum(dtype=torch.float64) for x in grads])
    return (scale * torch.sqrt(squares.sum())).float()


def _plain_clip(grads, outs, scale, most, limit):
    norm = _plain_norm(grads, scale, limit)
    factor = scale * torch.where(norm <= most, 1.0, most / norm)
    for x, o in zip(grads, outs):
        o.copy_(x.float() * factor)
    return norm


def _plain(s):
    op = s["op"]
    if op == "norm_forward":
        return _plain_norm_forward(s["x"], s["r"], s["gamma"], s["beta"])
    if op == "norm_backward":
        return _plain_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"], s["ds"], s["bias"])
    if op == "head_backward":
        return _plain_head_backward(s["h"], s["w"], s["target"], s["dlogp"], s["kept"])
    if op == "preference":
        return _plain_preference(s)
    if op == "policy":
        return _plain_policy(s)
    if op == "grad_norm":
        return _plain_norm(s["grads"], 1.0, s["limit"])
    return {"norm": _plain_clip(s["grads"], s["outs"], s["scale"], s["most"], s["limit"]), "grads": s["flat"]}


# ---------------------------------------------------------------- the package's operators

def _own(s):
    from spectral_corrected_optimizer_gb300 import finetune as ft
    op = s["op"]
    if op == "norm_forward":
        kept, x, y = ft.layer_norm(s["x"], s["r"], s["gamma"], s["beta"], EPS)
        return {"s": x, "y": y, "mean": kept.mean, "rstd": kept.rstd}
    if op == "norm_backward":
        kept = ft.NormStatistics(s["mean"], s["rstd"])
        dx, dgamma, dbeta = ft.layer_norm_backward(s["dy"], s["x"], kept, s["gamma"], ds=s["ds"], bias=s["bias"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta} if s["bias"] else {"dx": dx, "dgamma": dgamma}
    if op == "head_backward":
        dh, dw = ft.head_logp_backward(s["dlogp"], s["kept"], s["h"], s["w"], s["target"], ignore_index=IGNORE,
                                       dtype=torch.bfloat16)
        return {"dh": dh, "dw": dw}
    if op == "preference":
        loss, pair_loss, rewards, dlogp = ft.preference_loss(
            s["logp"], s["ref"], s["offsets"], beta=s["beta"], kind=s["kind"], smoothing=s["smoothing"],
            average=s["average"], mask=s["valid"])
        return {"loss": loss, "pair_loss": pair_loss, "rewards": rewards, "dlogp": dlogp}
    if op == "policy":
        loss, parts, dlogp = ft.policy_loss(
            s["logp"], s["old"], s["advantage"], s["offsets"], ref_logp=s["ref"], mask=s["valid"], clip_low=s["low"],
            clip_high=s["high"], kl_coef=s["kl"], reduction=s["reduction"])
        return {"loss": loss, "parts": parts, "dlogp": dlogp}
    if op == "grad_norm":
        return ft.grad_norm(s["grads"], norm_type=s["limit"])
    norm = ft.clip_grads(s["grads"], s["most"], scale=s["scale"], norm_type=s["limit"], out=s["outs"])
    return {"norm": norm, "grads": s["flat"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op = case["op"]
    if op in ("norm_forward", "norm_backward"):
        n, d, b = case["rows"], case["dim"], BYTES[case["type"]]
        forward = op == "norm_forward"
        tensors = (4 if case["residual"] else 2) if forward else (4 if case["residual"] else 3)
        vectors = (1 + case["bias"]) * d * b if forward else d * b + (1 + case["bias"]) * d * 4
        return {"bytes": tensors * n * d * b + 8 * n + vectors, "flops": (8 if forward else 14) * n * d}
    if op == "head_backward":
        n, v, d = case["tokens"], case["vocab"], case["dim"]
        kept = n * (1 - case["ignored"]) * (1 - case["still"])
        return {"bytes": 4 * (n * d + v * d) + (8 + 4 + 12) * n, "flops": 6 * kept * v * d}
    if op in ("preference", "policy"):
        count = 2 * case["pairs"] if op == "preference" else case["sequences"]
        n = int(_lengths(count, case["length"]).sum())
        tensors = 4 + 4 + 4 * case["reference"] + case["mask"]
        if op == "preference":
            return {"bytes": tensors * n + 8 * count + 6 * count, "flops": 4 * n}
        return {"bytes": (tensors + 4 + 4 * case["per_token"]) * n + 8 * count + 4 * count, "flops": 30 * n}
    n = _values(case)
    if op == "grad_norm":
        return {"bytes": n * BYTES[case["type"]], "flops": 2 * n}
    return {"bytes": n * (BYTES[case["type"]] + BYTES[case["out"]]), "flops": 3 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def _exact_norm_forward(s):
    x = s["x"].double()
    if s["r"] is not None:
        x = (x + s["r"].double()).to(s["x"].dtype).double()  # the stream is held in its own type
    dim = x.shape[1]
    mean = torch.einsum("nd->n", x) / dim
    variance = torch.einsum("nd,nd->n", x, x) / dim - mean * mean
    rstd = 1 / torch.sqrt(variance + EPS)
    y = torch.einsum("nd,n,d->nd", x - mean[:, None], rstd, s["gamma"].double())
    if s["beta"] is not None:
        y += s["beta"].double()
    return {"s": x, "y": y, "mean": mean, "rstd": rstd}


def _exact_norm_backward(s):
    dy, gamma, rstd, dim = s["dy"].double(), s["gamma"].double(), s["rstd"].double(), s["dim"]
    centred = s["x"].double() - s["mean"].double()[:, None]
    through = dy * gamma
    a = torch.einsum("nd->n", through) / dim
    b = torch.einsum("nd,nd->n", through, centred) * rstd ** 2 / dim
    dx = (through - a[:, None] - centred * b[:, None]) * rstd[:, None]
    if s["ds"] is not None:
        dx += s["ds"].double()
    out = {"dx": dx, "dgamma": torch.einsum("nd,nd,n->d", dy, centred, rstd)}
    return {**out, "dbeta": torch.einsum("nd->d", dy)} if s["bias"] else out


def _exact_head_backward(s):
    h, w, target, dlogp, kept = s["h"].double(), s["w"].double(), s["target"], s["dlogp"].double(), s["kept"].double()
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for rows in torch.nonzero((target != IGNORE) & (dlogp != 0))[:, 0].split(1024):
        d = torch.einsum("nd,vd->nv", h[rows], w)
        d *= math.log2(math.e)
        d -= kept[0, rows, None]
        d = torch.pow(2.0, d)
        d *= (-dlogp[rows] * kept[1, rows])[:, None]
        d[torch.arange(len(rows)), target[rows]] = dlogp[rows] * kept[2, rows]
        dh[rows] = d @ w
        dw.addmm_(d.T, h[rows])
    return {"dh": dh, "dw": dw}


def _span_sums(x, offsets):
    running = torch.cat((torch.zeros(1, dtype=torch.float64, device="cuda"), torch.cumsum(x, 0)))
    return running[offsets[1:]] - running[offsets[:-1]]


def _spread_spans(x, offsets, tokens):
    """A value per sequence at its tokens, 0 behind the last one."""
    out = torch.zeros(tokens, dtype=torch.float64, device="cuda")
    body = torch.repeat_interleave(x, offsets[1:] - offsets[:-1])
    out[:len(body)] = body
    return out


def _exact_preference(s):
    offsets, beta, eps, tokens = s["offsets"], s["beta"], s["smoothing"], len(s["logp"])
    x = s["logp"].double()
    if s["ref"] is not None:
        x = x - s["ref"].double()
    on = torch.ones_like(x) if s["valid"] is None else s["valid"].double()
    score = _span_sums(x * on, offsets)
    share = 1 / _span_sums(on, offsets).clamp_min(1) if s["average"] else torch.ones_like(score)
    score = score * share
    margin = beta * (score[0::2] - score[1::2])
    if s["kind"] == "logistic":
        loss = -(1 - eps) * torch.nn.functional.logsigmoid(margin) - eps * torch.nn.functional.logsigmoid(-margin)
        slope = -(1 - eps) * torch.sigmoid(-margin) + eps * torch.sigmoid(margin)
    elif s["kind"] == "hinge":
        loss, slope = torch.relu(1 - margin), torch.where(margin < 1, -1.0, 0.0).double()
    else:
        loss, slope = (margin / beta - 0.5 / beta) ** 2, 2 * (margin / beta - 0.5 / beta) / beta
    per = torch.empty_like(score)
    per[0::2], per[1::2] = slope, -slope
    dlogp = _spread_spans(per * share * beta / len(loss), offsets, tokens) * on
    return {"loss": loss.mean(), "pair_loss": loss, "rewards": (beta * score).view(-1, 2), "dlogp": dlogp}


def _exact_policy(s):
    offsets, tokens = s["offsets"], len(s["logp"])
    count = len(offsets) - 1
    logp = s["logp"].double()
    inside = _spread_spans(torch.ones(count, dtype=torch.float64, device="cuda"), offsets, tokens)
    on = inside if s["valid"] is None else inside * s["valid"].double()
    a = s["advantage"].double()
    if not s["per_token"]:
        a = _spread_spans(a, offsets, tokens)
    ratio = torch.exp(logp - s["old"].double())
    bounded = torch.where(a >= 0, ratio.clamp_max(1 + s["high"]), ratio.clamp_min(1 - s["low"]))
    out = bounded != ratio
    kl, dkl = torch.zeros_like(logp), torch.zeros_like(logp)
    if s["ref"] is not None:
        q = s["ref"].double() - logp
        kl, dkl = torch.exp(q) - q - 1, 1 - torch.exp(q)
    if s["reduction"] == "token":
        weight = on / on.sum().clamp_min(1)
    else:
        weight = on * _spread_spans(1 / _span_sums(on, offsets).clamp_min(1), offsets, tokens) / count
    parts = torch.stack([(weight * t).sum() for t in (-a * bounded, kl, out.double())])
    slope = torch.where(out, torch.zeros_like(a), -a * ratio) + s["kl"] * dkl
    return {"loss": parts[0] + s["kl"] * parts[1], "parts": parts, "dlogp": slope * weight}


def _exact_norm(grads, limit):
    if limit == math.inf:
        return max(float(x.abs().max()) for x in grads)
    return math.sqrt(math.fsum(float(torch.linalg.vector_norm(x, dtype=torch.float64)) ** 2 for x in grads))


def _exact_buffers(s, factor):
    """The clipped gradients, buffer by buffer, given back in 64 bits on the host where they are large."""
    place = "cpu" if _values(s) > 1 << 28 else "cuda"
    left = iter(s["grads"])
    return [torch.cat([(next(left).double() * factor).to(place) for _ in b]) for b in _sizes(s)]


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "norm_forward":
        return _exact_norm_forward(s)
    if op == "norm_backward":
        return _exact_norm_backward(s)
    if op == "head_backward":
        return _exact_head_backward(s)
    if op == "preference":
        return _exact_preference(s)
    if op == "policy":
        return _exact_policy(s)
    if op == "grad_norm":
        return torch.tensor(_exact_norm(s["grads"], case["limit"]), dtype=torch.float64)
    norm = case["scale"] * _exact_norm(s["grads"], case["limit"])
    factor = case["scale"] * min(1.0, s["most"] / norm)
    return {"norm": torch.tensor(norm, dtype=torch.float64), "grads": _exact_buffers(s, factor)}
