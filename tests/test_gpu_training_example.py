"""The operators together, as examples/prenorm_muon.py uses them: a rank's
gradients against torch's automatic differentiation of the same network in 64
bits, and the loss of a short training run."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_gradients_of_a_rank():
    import prenorm_muon
    net = prenorm_muon.Net(ranks=2, seed=3)
    x, t = net.batch()
    loss = float(net.rank_pass(1, x, t))
    f64 = lambda v: v.double().detach().requires_grad_()  # noqa: E731
    w1, w2 = f64(net.mats[0]["w"]), f64(net.mats[1]["w"])
    vec = f64(net.vec.lp[: net.plan.psi])

    def norm(i, h):
        mean, var = h.mean(1, keepdim=True), h.var(1, unbiased=False, keepdim=True)
        return (h - mean) / torch.sqrt(var + 1e-5) * net.vector(vec, i, 0) + net.vector(vec, i, 1)

    # relu's gates as the network set them: where rounding flips one, the two
    # derivatives have nothing to do with each other
    gates, low = [], x
    for i in range(net.layers):
        act = torch.relu(net.norm_forward(i, low)[0] @ net.mats[0]["w"][i].T)
        gates.append((act > 0).double())
        low = low + act @ net.mats[1]["w"][i].T
    h = x.double()
    for i in range(net.layers):
        h = h + ((norm(i, h) @ w1[i].T) * gates[i]) @ w2[i].T
    want = 0.5 * ((norm(net.layers, h) - t.double()) ** 2).sum(1).mean()
    want.backward()
    # every activation and gradient between the operators is rounded to bf16
    # (2^-9 of itself on average), a dozen of them in a row
    tol = 12 * 2.0 ** -9
    assert abs(loss - want.item()) <= tol * want.item()
    grads = net.vec.grads[1, : net.plan.psi]
    for got, ref in ((net.mats[0]["grads"][1], w1.grad), (net.mats[1]["grads"][1], w2.grad), (grads, vec.grad)):
        assert float((got.double() - ref).norm()) <= tol * float(ref.norm())
    assert not net.mats[0]["grads"][0].any()          # the other rank's buffers are its own


def test_training_lowers_the_loss():
    import prenorm_muon
    losses = prenorm_muon.train(steps=60, ranks=4)
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) < 0.7 * sum(losses[:5])
    assert losses == prenorm_muon.train(steps=60, ranks=4)      # the same bits every time
