"""The orthogonalised update and the Muon step over the whole range of fp32's
exponents.  Tolerances are those of test_gpu_muon; the norm's own rounding (a
compensated sum, a root and a division: under 1e-6) moves every singular value
by that much of itself, and five steps pass on at most five times that."""
import pytest
import torch

import zero_optimizer_step_02_gb300 as z
from test_gpu_muon import BF16, FP32, TORCH, gradients, orthogonalize, plain, tolerance

pytestmark = pytest.mark.gpu
NORM = 5e-6


def check(got, want, tol):
    for a, b in zip(got.double(), want):
        assert bool(torch.isfinite(a).all())
        assert float((a - b).norm()) <= tol * float(b.norm())


# either form (one SM's, the general one); sizes whose squares pass fp32's
# range at either end, beside an eps that matters and one that does not
@pytest.mark.parametrize("rows,cols", [(64, 64), (300, 520), (520, 300)])
@pytest.mark.parametrize("size,eps", [(1e-19, 1e-30), (1e-19, 1e-18), (1e-23, 1e-22), (2e-23, 1e-30), (1e-24, 1e-30),
                                      (1e-28, 1e-28), (1e-28, 1e-30), (1e13, 1e-7), (1e14, 1e-7), (1e20, 1e21), (5e37, 1e-7)])
@pytest.mark.parametrize("dt", [FP32, BF16])
def test_any_size_beside_any_eps(rows, cols, size, eps, dt):
    g = (100 * gradients(1, rows, cols)).clamp(-6.0, 6.0) * size
    x, o = orthogonalize(g, dt, FP32, 3, eps=eps)
    check(o, plain(x, eps=eps), tolerance(rows, cols, 3, FP32) + NORM)


def test_one_size_beside_another():
    # a few strong rows over a floor 2^60 below, and a floor alone in the others' batch
    g = 100 * gradients(3, 200, 300)
    g[0, 3:] *= 2.0 ** -60
    g[1] *= 2.0 ** -70
    x, o = orthogonalize(g, FP32, FP32, 3, eps=1e-30)
    check(o, plain(x, eps=1e-30), tolerance(200, 300, 3, FP32) + NORM)


def test_large_matrix_of_the_largest_values():
    # the norm itself passes fp32's range; a subnormal factor rounds the whole
    # of x_0 by up to 2^-18
    g = (100 * gradients(1, 1000, 1040)).clamp(-1.0, 1.0) * 3e38
    x, o = orthogonalize(g, FP32, FP32, 3)
    check(o, plain(x), tolerance(1000, 1040, 3, FP32) + NORM + 5 * 2.0 ** -18)


@pytest.mark.parametrize("rows,cols", [(64, 64), (300, 520)])
@pytest.mark.parametrize("size", [1e-20, 1e-24, 1e18])
def test_muon_of_a_matrix_whose_momentum_fades(rows, cols, size):
    d = z.matrices(rows, cols, eps=1e-30)
    grads = [torch.zeros(rows, cols, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    m = 100 * size * gradients(1, rows, cols)[0]
    w = gradients(1, rows, cols, 3)[0]
    lp = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    ws = torch.empty(z.zero_muon_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    sc = torch.zeros(256, dtype=torch.uint8, device="cuda")
    z.zero_scalars_init(sc)
    u, w0 = 0.9025 * m.double(), w.double()          # mu * (mu * m), mu = 0.95
    z.zero_muon_step(d, z.muon_hparams(lr=0.5), grads, m, w, lp, ws, sc)
    assert z.read_scalars(sc).status == 0
    # lr 0.5, no decay: what is added is half the orthogonalised direction
    o = plain(u[None], eps=1e-30)[0]
    off = float((w.double() - (w0 - 0.5 * o)).norm())
    assert off <= 0.5 * (tolerance(rows, cols, 3, FP32) + NORM + 2e-7) * float(o.norm()) + 2.0 ** -24 * float(w.double().norm())
    assert torch.equal(lp, w.to(TORCH[BF16]))
