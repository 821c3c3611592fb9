"""The join's backward pass reads the statistics of the norms that there are, and no others: a caller whose forward pass is
their own may leave the rest as they like."""
import pytest
import torch

from test_gpu_residual_norm import VECTORS, Case, z  # noqa: F401

pytestmark = pytest.mark.gpu


def results(c):
    rows = (c.dh, c.do) + ((c.dtok,) if c.dtok else ())
    return [r.v.clone() for r in rows] + [c.dw[k].clone() for k in VECTORS if c.dw[k] is not None]


@pytest.mark.parametrize("post,pre", [("none", "rms"), ("none", "layer"), ("rms", "none"), ("layer", "none"), ("rms", "rms"), ("layer", "rms"),
                                      ("rms", "layer"), ("none", "none")])
@pytest.mark.parametrize("gate", ["none", "vector", "token"])
@pytest.mark.parametrize("rows,cols,dt", [(50, 200, "bf16"), (20, 5000, "fp32"), (9, 1601, "fp16")])
def test_statistics_of_a_norm_that_is_not_there(z, post, pre, gate, rows, cols, dt):  # noqa: F811
    c = Case(z, rows, cols, dt, post=post, pre=pre, gate=gate, seed=21)
    c.forward()
    c.backward()
    c.check_backward()
    was = results(c)
    unread = [k for at, norm in ((0, post), (2, pre)) for k, read in ((at, norm == "layer"), (at + 1, norm != "none")) if not read]
    for other in (0.0, -3.0, float("inf"), float("nan")):
        c.stats[:, unread] = other
        c.backward()
        for got, want in zip(results(c), was):
            assert torch.equal(got, want), other
