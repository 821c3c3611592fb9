"""Clipping whose gradients are large, or not numbers: the norm of finite gradients is finite, and one that is not finite never
leaves a step unclipped."""
import numpy as np
import pytest
import torch

from test_gpu_adamw_tensors import F32, Tensor, run, scalars, z  # noqa: F401

pytestmark = pytest.mark.gpu


def large(rng, n, dtype, bits, size, shift):
    """Moments of a usual size under gradients of about `size`, among them elements of other sizes."""
    t = Tensor(rng, n, dtype, bits, shift=shift)
    g = t.d["grad"]
    g.copy_(torch.from_numpy(rng.standard_normal(n).astype(F32)).clamp(-3, 3) * size)
    g[:: 7] *= 2.0 ** -40
    t.before["grad"] = g.cpu().clone()
    return t


def norm_of(tensors):
    return float(np.sqrt(sum(np.sum(np.square(t.before["grad"].double().numpy())) for t in tensors)))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size", [3e18, 1e19, 1e25, 1e38])
def test_norm_of_large_gradients(z, dtype, bits, size):  # noqa: F811
    """Squares, or their sums, are past fp32's range; the coefficient is what 64 bits give."""
    rng = np.random.default_rng(41)
    hp = z.hparams(lr=1e-3, max_norm=1e3)
    ts = [large(rng, n, dtype, bits, size, shift) for n, shift in ((1, 0), (5000, 0), (2049, 1), (70_001, 0))]
    ts.append(Tensor(rng, 3000, dtype, bits))   # gradients of the usual size beside them
    sc = scalars(z)
    run(z, hp, ts, sc)
    got, norm = z.read_scalars(sc), norm_of(ts)
    assert abs(got.sqnorm - norm ** 2) <= 1e-12 * norm ** 2 and got.t == 1
    want = F32(1e3 / (norm + 1e-6))
    assert 0 < want < 1 and abs(int(F32(got.clip_coef).view(np.int32)) - int(want.view(np.int32))) <= 1
    for t in ts:
        t.check(hp, 0, coef=got.clip_coef, close=False)
        assert torch.isfinite(t.d["master"]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_of_a_few_large_gradients_among_many(z, dtype):  # noqa: F811
    """Tiles that are read four at a time: only some lanes' sums leave the range."""
    rng = np.random.default_rng(42)
    hp = z.hparams(lr=1e-3, max_norm=1.0)
    t = Tensor(rng, 12_000_123, dtype, 8)
    g = t.d["grad"]
    for at, x in ((5, 2e19), (6_000_000, -3e30), (6_000_007, 1e37), (12_000_122, 3e38)):
        g[at] = x
    t.before["grad"] = g.cpu().clone()
    sc = scalars(z)
    run(z, hp, [t], sc)
    got, norm = z.read_scalars(sc), norm_of([t])
    assert abs(got.sqnorm - norm ** 2) <= 1e-12 * norm ** 2
    want = F32(1.0 / (norm + 1e-6))
    assert abs(int(F32(got.clip_coef).view(np.int32)) - int(want.view(np.int32))) <= 1
    t.check(hp, 0, coef=got.clip_coef, close=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_norm_that_is_not_finite(z, dtype, bad, shift):  # noqa: F811
    """Without loss scaling: an infinite norm makes the coefficient 0, one that is no number NaN, as max_norm / norm says."""
    rng = np.random.default_rng(43)
    hp = z.hparams(lr=1e-3, max_norm=1.0, weight_decay=0.1)
    ts = [Tensor(rng, n, dtype, bits, shift=shift) for n, bits in ((5000, 32), (4097, 8), (300, 32))]
    ts[1].d["grad"][4000] = bad
    ts[1].before["grad"][4000] = bad
    sc = scalars(z)
    run(z, hp, ts, sc)
    got = z.read_scalars(sc)
    assert got.t == 1 and got.ctas_done == 0
    if np.isnan(bad):
        assert np.isnan(got.sqnorm) and np.isnan(got.clip_coef)
        assert all(torch.isnan(t.d["master"]).all() for t in ts)
    else:
        assert got.sqnorm == np.inf and got.clip_coef == 0.0
        assert all(torch.isfinite(t.d["master"]).all() for t in (ts[0], ts[2])) and int(torch.isnan(ts[1].d["master"]).sum()) == 1
    for t in ts:
        t.check(hp, 0, coef=got.clip_coef, close=False)


def test_large_gradients_under_loss_scaling(z):  # noqa: F811
    rng = np.random.default_rng(44)
    hp = z.hparams(lr=1e-3, max_norm=1.0, loss_scaling=True)
    ts = [large(rng, 5000, "fp32", bits, 1e30, 0) for bits in (32, 8)]
    sc = scalars(z, loss_scale=3.0)
    run(z, hp, ts, sc)
    got = z.read_scalars(sc)
    norm = np.sqrt(sum(np.sum(np.square((t.before["grad"].numpy() / F32(3)).astype(np.float64))) for t in ts))
    assert got.t == 1 and got.overflow == 0 and abs(got.sqnorm - norm ** 2) <= 1e-12 * norm ** 2
    for t in ts:
        t.check(hp, 0, coef=got.clip_coef, loss_scale=3.0, close=False)
