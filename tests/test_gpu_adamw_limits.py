"""The AdamW step with an eps at the bottom of fp32's range."""
import numpy as np
import pytest
import torch

from test_gpu_adamw_tensors import Tensor, run, scalars, z  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("eps", [1e-37, 1e-40])
def test_small_eps(z, eps, bits, shift):  # noqa: F811
    """eps * s is subnormal in the first steps: an element without a gradient stays where it is, one whose square is 0 is
    divided by eps * s, others as ever."""
    rng = np.random.default_rng(51)
    hp = z.hparams(lr=1e-3, eps=eps)
    t = Tensor(rng, 3 * 2048 + 300, "fp32", bits, lp=None, shift=shift)
    for k in ("m", "v", "m_scale", "v_scale"):
        if k in t.d:
            t.d[k].zero_()
    g = t.d["grad"]
    g[::3] = 0.0
    g[1::3] *= 1e-24   # squares underflow
    t.before = {k: x.cpu().clone() for k, x in t.d.items()}
    run(z, hp, [t], scalars(z))
    t.check(hp, 0, close=False)
    assert torch.equal(t.d["master"][::3].cpu(), t.before["master"][::3]) and not torch.isnan(t.d["master"]).any()
