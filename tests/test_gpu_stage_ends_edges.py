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
