"""A small pre-norm network trained with every operator of the library's
training side: layer norm forward and backward, the Muon step for the weight
matrices, the ZeRO-DP Adam step for the norm vectors.

    python examples/prenorm_muon.py [--steps 60] [--ranks 4]

N_d data-parallel ranks are simulated on one GPU, as everywhere in this
library: each rank runs its own micro-batch forward and backward and leaves
16-bit gradients in its own flat buffers; `zero_layernorm_backward` writes the
norms' weight gradients straight into them.  The optimizer calls reduce over
the ranks:
  - matrices:  zero_muon_step    (rank mean, momentum, orthogonalised update)
  - vectors:   zero_step_fused   (rank mean, Adam, gather)
The matrix products of the network itself are plain torch.

    h_0 = x;  h_{l+1} = h_l + W2_l relu(W1_l norm_l(h_l));  y = norm_L(h_L)
    loss = sum over features of (y - target)^2 / 2, mean over tokens
"""
import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import zero_optimizer_step_02_gb300 as z  # noqa: E402


class Net:
    """Parameters, optimizer state and one set of gradient buffers a rank."""

    def __init__(self, layers=2, width=256, hidden=512, tokens=512, ranks=4, seed=0):
        self.layers, self.width, self.hidden, self.tokens, self.ranks = layers, width, hidden, tokens, ranks
        dev, bf16 = "cuda", torch.bfloat16
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
        # vectors: gain and bias of each norm, one flat space for the Adam step
        self.norms = layers + 1
        self.adam = z.hparams(lr=3e-3)
        self.plan = z.Plan(2 * self.norms * width, ranks, stage=2)
        self.vec = z.StepBuffers(self.plan, self.adam)
        self.vec.master[: self.plan.psi].view(self.norms, 2, width)[:, 0] = 1.0
        self.vec.lp.copy_(self.vec.master[: self.plan.psi])
        self.vec.init_scalars()
        # matrices: W1 [hidden, width] and W2 [width, hidden], one batch of each
        self.muon = z.muon_hparams(lr=1e-2, momentum=0.95, rms_scale=0.2)
        self.mats = []
        for rows, cols in ((hidden, width), (width, hidden)):
            d = z.matrices(rows, cols, batch=layers)
            master = rnd(layers, rows, cols) * cols ** -0.5
            self.mats.append(dict(
                desc=d, master=master, momentum=torch.zeros_like(master), w=master.to(bf16),
                grads=[torch.zeros(layers, rows, cols, device=dev, dtype=bf16) for _ in range(ranks)],
                ws=torch.empty(z.zero_muon_workspace_bytes(d), dtype=torch.uint8, device=dev)))
        self.ln = z.layernorm(tokens, width, dtype=z.ZERO_BF16, w_dtype=z.ZERO_BF16)
        self.ln_ws = torch.empty(z.zero_layernorm_workspace_bytes(self.ln), dtype=torch.uint8, device=dev)
        self.teacher = rnd(width, width) * width ** -0.5
        self.rnd = rnd

    def batch(self):
        """One micro-batch: inputs and the (normalised) targets of a fixed teacher."""
        x = self.rnd(self.tokens, self.width)
        t = torch.tanh(x @ self.teacher)
        t = (t - t.mean(1, keepdim=True)) / t.std(1, keepdim=True)
        return x.to(torch.bfloat16), t

    def vector(self, flat, norm, which):
        """gain (0) or bias (1) of a norm in a flat vector buffer."""
        at = (2 * norm + which) * self.width
        return flat[at: at + self.width]

    def norm_forward(self, i, x):
        y, mean, rstd = torch.empty_like(x), torch.empty(len(x), device="cuda"), torch.empty(len(x), device="cuda")
        z.zero_layernorm_forward(self.ln, x, self.vector(self.vec.lp, i, 0), self.vector(self.vec.lp, i, 1), y, mean, rstd)
        return y, (x, mean, rstd)

    def norm_backward(self, i, dy, saved, rank):
        x, mean, rstd = saved
        dx = torch.empty_like(x)
        grads = self.vec.grads[rank]
        z.zero_layernorm_backward(self.ln, dy.contiguous(), x, self.vector(self.vec.lp, i, 0), mean, rstd, dx,
                                  self.vector(grads, i, 0), self.vector(grads, i, 1), self.ln_ws)
        return dx

    def rank_pass(self, rank, x, target):
        """Forward and backward of one rank's micro-batch; its loss (a device tensor)."""
        w1, w2 = self.mats[0]["w"], self.mats[1]["w"]
        h, saved = x, []
        for i in range(self.layers):
            y, s = self.norm_forward(i, h)
            a = torch.relu(y @ w1[i].T)
            saved.append((s, y, a))
            h = h + a @ w2[i].T
        y, s = self.norm_forward(self.layers, h)
        err = y.float() - target
        loss = 0.5 * (err * err).sum(1).mean()
        dh = self.norm_backward(self.layers, (err / self.tokens).to(torch.bfloat16), s, rank)
        for i in reversed(range(self.layers)):
            s, y, a = saved[i]
            self.mats[1]["grads"][rank][i] = dh.T @ a
            da = (dh @ w2[i]) * (a > 0)
            self.mats[0]["grads"][rank][i] = da.T @ y
            dh = dh + self.norm_backward(i, da @ w1[i], s, rank)
        return loss

    def optimize(self):
        for m in self.mats:
            z.zero_muon_step(m["desc"], self.muon, m["grads"], m["momentum"], m["master"], m["w"], m["ws"], self.vec.scalars)
        self.vec.step(self.adam)

    def step(self):
        loss = sum(self.rank_pass(r, *self.batch()) for r in range(self.ranks)) / self.ranks
        self.optimize()
        return loss


def train(steps=60, ranks=4, seed=0, every=0):
    """Losses of `steps` training steps; prints one of `every`."""
    net = Net(ranks=ranks, seed=seed)
    losses = []
    for k in range(steps):
        losses.append(net.step())
        if every and k % every == 0:
            print("step %3d  loss %.3f" % (k, float(losses[-1])))
    losses = torch.stack(losses).tolist()
    status = net.vec.scalars_host().status
    if status:
        raise RuntimeError("a device wait ran out (status %d)" % status)
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--ranks", type=int, default=4)
    a = ap.parse_args()
    got = train(a.steps, a.ranks, every=10)
    print("loss %.3f -> %.3f" % (got[0], got[-1]))
