"""8-bit states whose tiles go through the ring, which carries on from one tensor to the next."""
import numpy as np
import pytest
import torch

from test_gpu_adamw_tensors import Tensor, run, scalars, z  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("clip", [False, True])
def test_ring_over_many_tensors(z, clip):  # noqa: F811
    """Twelve tiles a CTA over several tensors, with others between them that do not take the ring; the ring wraps within
    a tensor and goes on in the next."""
    rng = np.random.default_rng(61)
    hp = z.hparams(lr=1e-3, beta2=0.95, weight_decay=0.1, max_norm=0.5 if clip else 0.0)
    kinds = [("bf16", 8, 0), ("fp32", 8, 0), ("bf16", 32, 0), ("fp16", 8, 0), ("fp32", 8, 1)]
    ts = [Tensor(rng, int(rng.integers(3, 26)) * 2048 + int(rng.integers(0, 2048)) * (k % 3 != 0), *kinds[k % 5][:2], lp=["bf16", "fp16", None][k % 3],
                 shift=kinds[k % 5][2], wd_scale=float(k % 2), lr_scale=0.5 + k % 3) for k in range(400)]
    assert sum(-(-t.n // 2048) for t in ts) >= 10 * 456
    sc = scalars(z, 3, hp)
    run(z, hp, ts, sc)
    got = z.read_scalars(sc)
    assert got.t == 4 and got.status == 0
    for t in ts:
        t.check(hp, 3, coef=got.clip_coef if clip else None, close=False)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lp", ["bf16", "fp16"])
def test_narrow_weights_beside_one_that_is_not_a_number(z, bits, lp):  # noqa: F811
    """The 16-bit weights are the cast of the weights, element by element."""
    rng = np.random.default_rng(62)
    hp = z.hparams(lr=1e-3)
    t = Tensor(rng, 5003, "fp32", bits, lp)
    for at in (0, 2100, 5002):
        t.d["grad"][at] = float("nan")
    t.before["grad"] = t.d["grad"].cpu().clone()
    run(z, hp, [t], scalars(z))
    t.check(hp, 0, close=False)
    p, got = t.d["master"], t.d["lp"]
    nan = torch.isnan(p)
    assert int(nan.sum()) == 3 and torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], p[~nan].to(got.dtype))
