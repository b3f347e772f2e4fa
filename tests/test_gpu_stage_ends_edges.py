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
