"""The stage-end operators at the edges of what their header promises, against
the float64 forms of stage_ends_ref.py.  Tolerances are those derived in
test_gpu_stage_ends.py unless a test derives its own."""
import pytest
import torch

import stage_ends_ref as ref
import test_gpu_stage_ends as base
from gpu_util import ensure_lib

pytestmark = pytest.mark.gpu

U32, BF, FP = base.U32, base.BF, base.FP


@pytest.fixture(scope="module", autouse=True)
def _lib():
    ensure_lib()


@pytest.fixture(autouse=True)
def _clean_flag(_lib):
    yield
    import spectral_corrected_optimizer_gb300 as so
    so.check_device()


# ---------------------------------------------------------------- residual norm: the widest rows

@pytest.mark.parametrize("dim", [32761, 32762, 32763, 32767])
@pytest.mark.parametrize("rows", [1, 9])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_of_the_widest_odd_rows(rows, dim, dtype):
    base.test_residual_norm_and_its_backward(rows, dim, dtype, True)


@pytest.mark.parametrize("dim", [32760, 32768])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_of_the_widest_rows_off_a_boundary(dim, dtype):
    x, r, gamma, g = base.norm_inputs(5, dim, dtype, True, seed=2)
    sh, op = base.shifted, base.se()
    kept, s, y = op.residual_norm(sh(x, 1), sh(r, 3), sh(gamma, 2), 1e-5)
    want_s = (x.float() + r.float()).to(dtype)
    q, scale = ref.checkpoint32(want_s)
    assert torch.equal(s.cpu(), want_s) and torch.equal(kept.scale.cpu(), scale)
    assert torch.equal(kept.q.cpu().view(torch.uint8), q.view(torch.uint8))
    want_y, rstd = ref.norm_forward(want_s, gamma, 1e-5)
    assert bool(((kept.rstd.cpu().double() - rstd).abs() <= 100 * U32 * rstd).all())
    assert bool(((y.cpu().double() - want_y).abs() <= (base.u_of(dtype) + 104 * U32) * want_y.abs()).all())
    dy = base.randn(g, x.shape, dtype)
    dx, dgamma, y2 = op.residual_norm_backward(sh(dy, 3), kept, sh(gamma, 1), ds=sh(r, 2), recompute=True)
    w = ref.norm_backward(dy, r, kept.q.cpu(), kept.scale.cpu(), kept.rstd.cpu(), gamma)
    assert bool(((dx.cpu().double() - w[0]).abs() <= base.u_of(dtype) * w[0].abs() + 100 * U32 * w[1]).all())
    assert bool(((dgamma.cpu().double() - w[2]).abs() <= 15 * U32 * w[3]).all())
    assert bool(((y2.cpu().double() - w[4]).abs() <= (base.u_of(dtype) + 4 * U32) * w[4].abs()).all())


# ---------------------------------------------------------------- head: logits that are not finite

@pytest.mark.parametrize("others", [0.0, -200.0, 150.0])
def test_head_of_an_impossible_target(others):
    # token 0: the target's logit overflows to -inf, the 599 other logits are equal; token 1 is an ordinary one
    vocab, dim = 600, 16
    w, h = torch.zeros(vocab, dim, dtype=BF), torch.zeros(2, dim, dtype=BF)
    h[0, 0], h[0, 1], h[1, 2] = 3e38, 1.0, 1.0
    w[:, 1] = others
    w[7, 0] = -1000.0
    w[:, 2] = torch.linspace(-2, 2, vocab).to(BF)
    target = torch.tensor([7, 80])
    args = h.cuda(), w.cuda(), target.cuda()
    loss, row_loss, dh, dw = base.se().head_loss_grad(*args)
    assert float(row_loss[0]) == float("inf") and float(loss) == float("inf")
    want = ref.head(h[1:], w, target[1:])
    base.check_loss(row_loss[1], row_loss[1:], want, dim)
    # softmax - onehot of token 0: -1 at its target, 1 / 599 elsewhere, rounded to bf16; half of it for the mean
    p = torch.full((vocab,), 1 / 599, dtype=torch.float64)
    p[7] = -1.0
    assert bool(((dw[:, 1].cpu().double() - p / 2).abs() <= base.U16 * p.abs() / 2).all())
    assert bool(dw.isfinite().all()) and bool(dh.isfinite().all())
    assert torch.equal(base.se().head_loss(*args)[1], row_loss)


def test_head_of_a_finite_loss_beyond_1e38():
    # lse = log(3 + 0), the target's logit is -2.5e38: finite in e, beyond fp32 in log2
    w, h = torch.zeros(4, 8, dtype=BF), torch.zeros(1, 8, dtype=BF)
    h[0, 0], w[2, 0] = 2.5e38, -1.0
    row_loss = base.se().head_loss(h.cuda(), w.cuda(), torch.tensor([2]).cuda())[1]
    assert abs(float(row_loss[0]) / float(h[0, 0]) - 1) <= 4 * U32
    # an infinite target's logit and other rows' NaN stay visible
    w[2, 0] = 1e3
    assert bool(base.se().head_loss(h.cuda(), w.cuda(), torch.tensor([2]).cuda())[1].isnan().all())


# ---------------------------------------------------------------- head: large logits

def test_head_probabilities_of_large_logits():
    # all 512 logits of token i are L_i, exactly: every probability is 2^-9, which bf16 holds, and an error of
    # 2^-10 of it (a rounding of fp32 at 1.44 L_i from L_i = 3e4 on) would come out as another value
    large = torch.tensor([3.0e4, -4.3e4, 6.1e4, -9.9e4, 2.3e5, -3.3e5, 7.7e5, 1.1e6], dtype=BF)
    n, vocab, dim = len(large), 512, 16
    h, w = torch.zeros(n, dim, dtype=BF), torch.zeros(vocab, dim, dtype=BF)
    h[:, :n] = torch.diag(large)
    w[:, :n] = 1.0
    target = torch.arange(n) * 60
    row_loss, dw = [base.se().head_loss_grad(h.cuda(), w.cuda(), target.cuda())[i].cpu() for i in (1, 3)]
    want = (large.float() / vocab / n).expand(vocab, n).clone()
    want[target, torch.arange(n)] = 0
    got = dw[:, :n].clone()
    got[target, torch.arange(n)] = 0
    assert torch.equal(got, want)
    onto = dw[target, torch.arange(n)].double() / large.double() * n
    assert bool(((onto + 511 / 512).abs() <= base.U16).all()) and bool(row_loss.isfinite().all())


# ---------------------------------------------------------------- head: what a logit's sum may lose
#
# A row's logits other than the target's carry the tensor cores' truncation, of which the mean over normal values
# (0.38 to 0.54 times UNIT(dim) of the logit) is given back as half a unit.

def unit(dim):
    return 2.0 ** -24 * dim / 32


def loss_error(h, w, target):
    """(error of row_loss, the float64 loss, lse, largest magnitude of a row's logits)."""
    row = base.se().head_loss(h.cuda(), w.cuda(), target.cuda())[1].double()
    logits = h.cuda().double() @ w.cuda().double().T
    lse = torch.logsumexp(logits, 1)
    want = lse - logits.gather(1, target.cuda()[:, None])[:, 0]
    return (row - want).cpu(), want.cpu(), lse.cpu(), logits.abs().amax(1).cpu()


@pytest.mark.parametrize("dim,held", [(4096, 1), (4096, 3), (65536, 1), (2056, 2)])
@pytest.mark.parametrize("tokens", [40, 700])
def test_head_keeps_exact_sums_of_a_few_values(tokens, dim, held):
    # `held` values of h per token that are not 0, whole numbers of 8 bits in w: every sum is exact, so what is left are
    # the exponents' factor (2^-24 of it, and 2^-26 per group of 16 values behind the first) and exp and log
    g, vocab = base.gen(dim + held), 300
    h, w = torch.zeros(tokens, dim, dtype=BF), torch.randint(-255, 256, (vocab, dim), generator=g).to(BF)
    for _ in range(held):
        h[torch.arange(tokens), torch.randint(0, dim, (tokens,), generator=g)] = 1.0
    err, _, lse, most = loss_error(h, w, torch.randint(0, vocab, (tokens,), generator=g))
    assert bool((err.abs() <= 2.0 ** -23 * most + 2.0 ** -22 * (lse.abs() + 8)).all()), float(err.abs().max())


@pytest.mark.parametrize("dim", [2048, 4096])
def test_head_bounds_the_error_of_exact_dense_sums(dim):
    g, tokens, vocab = base.gen(dim), 200, 300
    h = torch.randint(-3, 4, (tokens, dim), generator=g).to(BF)
    w = (torch.randint(-2, 3, (vocab, dim), generator=g) * 0.5).to(BF)
    err, _, lse, most = loss_error(h, w, torch.randint(0, vocab, (tokens,), generator=g))
    assert bool((err.abs() <= (unit(dim) / 2 + 2.0 ** -23) * most + 2.0 ** -22 * (lse.abs() + 8)).all())


@pytest.mark.parametrize("dim", [2048, 4096])
@pytest.mark.parametrize("common", [True, False])
def test_head_gives_the_mean_truncation_back(dim, common):
    # common: all rows of w point the same way, so that all logits of a token are near one another and the loss shows
    # the truncation of their common part; otherwise one logit of size 50 stands out over 0s
    g, tokens, vocab = base.gen(dim), 2048, 512
    r = torch.randn(dim, generator=g)
    h = torch.randn(tokens, dim, generator=g)
    if common:
        r *= 20 / dim ** 0.5
        h += 2.5 * r / r.norm()
        w = (r + 0.02 * torch.randn(vocab, dim, generator=g)).to(BF)
        target = torch.randint(0, vocab, (tokens,), generator=g)
    else:
        w = torch.zeros(vocab, dim, dtype=BF)
        w[1] = r * 60 / dim ** 0.5
        target = torch.zeros(tokens, dtype=torch.int64)
    h = h.to(BF)
    err, want, lse, _ = loss_error(h, w, target)
    rows = lse > 25
    assert int(rows.sum()) > 500
    rel = (err / lse)[rows] / unit(dim)
    # the mean: 0.12 units, and four deviations of 0.4 / sqrt(rows); a missing or doubled factor leaves 0.4 or more
    assert abs(float(rel.mean())) <= 0.12 + 1.6 / int(rows.sum()) ** 0.5
    assert float(rel.square().mean().sqrt()) <= 0.5


def test_head_loss_of_well_predicted_tokens_keeps_its_digits():
    # the target's logit is 8 to 60, the 599 others 0: loss = log(1 + 599 e^-l), down to 5e-24
    vocab, tokens = 600, 14
    h, w = torch.zeros(tokens, 64, dtype=BF), torch.zeros(vocab, 64, dtype=BF)
    h[:, 0], w[5, 0] = torch.arange(8, 64, 4).to(BF), 1.0
    row, dw = [base.se().head_loss_grad(h.cuda(), w.cuda(), torch.full((tokens,), 5).cuda(), reduction="sum")[i].cpu().double()
               for i in (1, 3)]
    want = torch.log1p(599 * torch.exp(-h[:, 0].double()))
    # the exponent is off by 2^-23 of the logit at most, exp, log1p and the sum of 600 terms by 2^-20
    assert bool(((row / want - 1).abs() <= 2.0 ** -23 * h[:, 0].double() + 2.0 ** -20).all())
    assert abs(float(dw[5, 0]) / float(-((1 - torch.exp(-want)) * h[:, 0].double()).sum()) - 1) <= base.U16


# ---------------------------------------------------------------- residual norm in place

def entry(name, *args):
    """A C entry point called on the current stream, tensors as their pointers."""
    import spectral_corrected_optimizer_gb300 as so
    ptr = lambda a: a.data_ptr() if isinstance(a, torch.Tensor) else a  # noqa: E731
    so._check(getattr(so.lib(), name)(*map(ptr, args), torch.cuda.current_stream().cuda_stream), name)


# rows: more than blocks; widths: one, two (a ring of rows in the backward pass), eight and nine pieces per thread
@pytest.mark.parametrize("rows,dim", [(10000, 64), (10000, 67), (1300, 2048), (1300, 2051), (700, 8200), (330, 16400),
                                      (330, 16403), (160, 32766)])
@pytest.mark.parametrize("by", [0, 1])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_norm_in_place(rows, dim, by, dtype):
    g, op = torch.Generator("cuda").manual_seed(rows + dim), base.se()
    code, eps = (0 if dtype == BF else 1), 1e-5
    x, r, dy, ds = [base.shifted(torch.randn(rows, dim, generator=g, device="cuda").to(dtype), by) for _ in range(4)]
    gamma = base.shifted(torch.randn(dim, generator=g, device="cuda").to(dtype), by)
    q = base.shifted(torch.zeros(rows, dim, dtype=torch.uint8), by)
    y, scale, rstd = torch.empty_like(x), torch.empty(rows, -(-dim // 128), device="cuda"), torch.empty(rows, device="cuda")
    kept, s, want_y = op.residual_norm(x, r, gamma, eps)
    for over in (0, 1):
        pair = [base.shifted(t, by) for t in (x, r)]
        entry("resnorm_forward", *pair, gamma, code, eps, pair[over], y, q, scale, rstd, rows, dim)
        assert torch.equal(pair[over], s) and torch.equal(pair[1 - over], (x, r)[1 - over]) and torch.equal(y, want_y)
        assert torch.equal(q, kept.q.view(torch.uint8)) and torch.equal(scale, kept.scale) and torch.equal(rstd, kept.rstd)
    import spectral_corrected_optimizer_gb300 as so
    ws = torch.empty(so.lib().resnorm_backward_workspace(rows, dim), dtype=torch.uint8, device="cuda")

    def backward(dy, ds, dx):  # dx begins where dy and ds do: its place decides how a row's sums are grouped
        dgamma = torch.empty(dim, device="cuda")
        entry("resnorm_backward", dy, ds, q, scale, rstd, gamma, code, dx, dgamma, y, rows, dim, ws, ws.numel())
        return dx, dgamma, y.clone()

    want = backward(dy, ds, base.shifted(torch.zeros_like(x), by))
    for over in (0, 1):
        pair = [base.shifted(t, by) for t in (dy, ds)]
        assert all(torch.equal(a, b) for a, b in zip(backward(*pair, pair[over]), want))


# ---------------------------------------------------------------- embedding gradient: long lists, large vocabularies

@pytest.mark.parametrize("tokens,vocab,dim,passes", [(5000, 300, 8, 1), (70000, 200000, 16, 2), (70000, 300000, 16, 3),
                                                     (262144 + 5, 300000, 8, 3), (1200001, 1000, 3, 2),
                                                     (1200001, 300000, 8, 3), (300000, 2 ** 27 + 3, 1, 4)])
def test_embed_grad_of_many_tiles_and_passes(tokens, vocab, dim, passes):
    # several tiles of 2048 tokens, 9 bits of the ids a pass; from 128 tiles on their counts are scanned by a launch
    assert (vocab.bit_length() + 8) // 9 == passes
    g = base.gen(tokens + vocab)
    ids = torch.where(torch.rand(tokens, generator=g) < 0.5, base.zipf(g, tokens, vocab),
                      torch.randint(0, vocab, (tokens,), generator=g))
    dy = base.randn(g, (tokens, dim), BF)
    grad = base.se().embed_grad(ids.cuda(), dy.cuda(), vocab)
    some, at = ids.unique(return_inverse=True)
    base.check_grad(grad[some.cuda()], at, dy, len(some), 1.0)
    grad[some.cuda()] = 0
    assert not bool(grad.any())


def test_embed_grad_grows_with_the_tokens_not_with_their_square():
    def best(tokens):
        ids = torch.randint(0, 5000, (tokens,), device="cuda")
        dy, out = torch.ones(tokens, 1, dtype=BF, device="cuda"), torch.empty(5000, 1, device="cuda")
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            base.se().embed_grad(ids, dy, 5000, out=out)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    # 32 times the tokens; with a pass that grew with their square it was over 90 times the time
    assert best(2 ** 25) < 50 * best(2 ** 20)


# ---------------------------------------------------------------- head: many tokens

@pytest.mark.parametrize("tokens", [65535, 65536, 70001, 150000])
@pytest.mark.parametrize("idt", [torch.int64, torch.int32])
def test_head_of_many_tokens(tokens, idt):
    # from 65536 tokens on a launch of its own counts the targets of whole stretches of 4096
    g, vocab, dim = base.gen(tokens), 40, 8
    h, w = base.randn(g, (tokens, dim), BF), base.randn(g, (vocab, dim), BF)
    target = torch.randint(0, vocab, (tokens,), generator=g, dtype=idt)
    target[torch.rand(tokens, generator=g) < 0.3] = -100
    target[4096:12288] = -100
    loss, row_loss, dh, dw = base.se().head_loss_grad(h.cuda(), w.cuda(), target.cuda())
    want = ref.head(h, w, target)
    base.check_loss(loss, row_loss, want, dim)
    base.check_grads(dh, dw, want, h, w)
    only = base.se().head_loss(h.cuda(), w.cuda(), target.cuda())
    assert torch.equal(only[0], loss) and torch.equal(only[1], row_loss)


def test_head_grows_with_the_tokens_not_with_their_square():
    def best(tokens):
        target = torch.randint(0, 8, (tokens,), device="cuda")
        h, w = torch.ones(tokens, 8, dtype=BF, device="cuda"), torch.ones(8, 8, dtype=BF, device="cuda")
        times = []
        for _ in range(4):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            base.se().head_loss(h, w, target)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    # 32 times the tokens; counting targets with their square it was over 200 times the time
    assert best(2 ** 23) < 50 * best(2 ** 18)


# ---------------------------------------------------------------- reports

def test_check_device_costs_little_more_than_one_read():
    import time

    import spectral_corrected_optimizer_gb300 as so

    def best(f):
        times = []
        for _ in range(400):
            t = time.perf_counter()
            f()
            times.append(time.perf_counter() - t)
        return min(times)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    # both flags in one synchronisation: 1.3 reads of a word; one after the other they took 2
    assert best(so.check_device) < 1.7 * best(word.item)


def test_reports_of_ids_come_once_and_in_any_thread():
    import threading

    import spectral_corrected_optimizer_gb300 as so
    table, ids = torch.ones(4, 8, device="cuda"), torch.tensor([9], device="cuda")
    errors = []

    def check():
        try:
            so.check_device()
        except so.SpecOptimError as e:
            errors.append(e.code)
    for _ in range(2):
        base.se().embed_lookup(table, ids)
        torch.cuda.synchronize()
        for t in [threading.Thread(target=check) for _ in range(3)]:
            t.start()
            t.join()
    assert errors == [so.ERR_BOUNDS] * 2
