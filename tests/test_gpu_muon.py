"""The orthogonalised update and the Muon step on the GPU against plain
evaluations in 64 bits.

Tolerances (relative, 2-norm of the difference over that of the result), from
the arithmetic.  One product: every operand is rounded to fp16, 2e-4 root mean
square, and a step passes on about five such errors (x and P in P x, x twice in
the Gram matrix, G in G G); five steps that add up coherently, the worst case
(a single row), make 6e-3.  Three products: operands of 22 bits, and an
accumulator that loses up to 2^-23 of itself at each addition of a 16-deep
slice: 5 * (2e-6 + depth / 16 * 2^-23).  The result's own rounding comes on
top.  An element may be off by eight times the root mean square error allowed."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_02_gb300 as z

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = z.ZERO_BF16, z.ZERO_FP16, z.ZERO_FP32
TORCH = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32}
UNIT = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
QUINTIC = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def plain(g, steps=5, coefs=None, eps=EPS):
    x = g.double()
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.transpose(-1, -2)
    x = x / (x.norm(dim=(-2, -1), keepdim=True) + eps)
    for a, b, c in (coefs or [QUINTIC] * steps):
        gram = x @ x.transpose(-1, -2)
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.transpose(-1, -2) if tall else x


def tolerance(rows, cols, products, out_dt):
    depth = max(rows, cols)
    return (6e-3 if products == 1 else 5 * (2e-6 + depth / 16 * 2.0 ** -23)) + UNIT[out_dt]


def gradients(batch, rows, cols, seed=0):
    g = torch.Generator().manual_seed(seed * 7919 + batch * 31 + rows * 3 + cols)
    k = max(1, min(rows, cols) // 16)
    low = torch.randn(batch, rows, k, generator=g) @ torch.randn(batch, k, cols, generator=g) / k ** 0.5
    return (1e-2 * (low + torch.randn(batch, rows, cols, generator=g))).cuda()


def check(got, want, tol):
    d = (got.double() - want)
    for i in range(want.shape[0]):
        rms = float(want[i].norm()) / want[i].numel() ** 0.5
        assert float(d[i].norm()) <= tol * float(want[i].norm())
        assert float(d[i].abs().max()) <= 8 * tol * max(rms, float(want[i].abs().max()))


def orthogonalize(g, dt, out_dt, products=0, ld=0, out_ld=0, gap=0, **kw):
    """g: [batch, rows, cols]; ld / out_ld: row strides, gap: elements between matrices; guarded by NaN."""
    b, r, c = g.shape
    ld, old = ld or c, out_ld or c
    si, so = r * ld + gap, r * old + gap
    src = torch.full((b * si + 8,), float("nan"), dtype=TORCH[dt], device="cuda")
    dst = torch.full((b * so + 8,), float("nan"), dtype=TORCH[out_dt], device="cuda")
    view = lambda t, s, l: torch.as_strided(t, (b, r, c), (s, l, 1))  # noqa: E731
    view(src, si, ld).copy_(g.to(TORCH[dt]))
    d = z.matrices(r, c, batch=b, dtype=dt, out_dtype=out_dt, in_ld=ld, out_ld=old, stride=si, out_stride=so,
                   products=products, **kw)
    ws = torch.full((z.zero_orthogonalize_workspace_bytes(d),), 0xFF, dtype=torch.uint8, device="cuda")
    sc = torch.zeros(256, dtype=torch.uint8, device="cuda")
    z.zero_scalars_init(sc)
    z.zero_orthogonalize(d, src, dst, ws, sc)
    assert z.read_scalars(sc).status == 0
    out = view(dst, so, old).clone()
    view(dst, so, old).fill_(float("nan"))
    assert bool(torch.isnan(dst).all())          # nothing written around the matrices
    return view(src, si, ld), out


SHAPES = [(1, 1, 1), (1, 1, 7), (1, 9, 1), (1, 2, 3), (1, 17, 33), (2, 63, 64), (1, 65, 64), (3, 127, 129), (1, 96, 160),
          (1, 128, 128), (2, 129, 255), (1, 256, 257), (1, 333, 1601), (1, 511, 385), (1, 768, 768), (5, 300, 700),
          (40, 300, 700), (40, 700, 301), (10, 513, 520), (60, 130, 258), (1, 1300, 1290)]


@pytest.mark.parametrize("products", [1, 3])
@pytest.mark.parametrize("batch,rows,cols", SHAPES)
def test_shapes(batch, rows, cols, products):
    g = gradients(batch, rows, cols)
    x, o = orthogonalize(g, FP32, FP32, products)
    check(o, plain(x), tolerance(rows, cols, products, FP32))


# either side of the form that keeps a matrix in one SM (128 x 256), more
# matrices than SMs, every width of its panels
@pytest.mark.parametrize("batch,rows,cols", [(1, 128, 256), (1, 256, 128), (1, 129, 256), (1, 256, 129), (1, 128, 257),
                                             (1, 257, 128), (200, 64, 64), (170, 20, 250), (3, 1, 256), (3, 256, 1),
                                             (1, 16, 16), (1, 15, 17), (2, 113, 65), (2, 191, 127), (1, 100, 193)])
def test_small_shapes(batch, rows, cols):
    g = gradients(batch, rows, cols)
    x, o = orthogonalize(g, FP32, FP32, 3)
    check(o, plain(x), tolerance(rows, cols, 3, FP32))


@pytest.mark.parametrize("dt,out_dt", [(BF16, BF16), (FP16, FP16), (FP32, BF16), (BF16, FP32), (FP32, FP16)])
@pytest.mark.parametrize("batch,rows,cols,ld,old,gap", [(2, 96, 160, 0, 0, 0), (2, 96, 160, 168, 176, 8), (3, 130, 77, 0, 0, 0),
                                                        (3, 130, 77, 81, 79, 5), (1, 64, 513, 520, 513, 0)])
def test_types_and_strides(batch, rows, cols, ld, old, gap, dt, out_dt):
    x, o = orthogonalize(gradients(batch, rows, cols), dt, out_dt, 0, ld, old, gap)
    check(o, plain(x), tolerance(rows, cols, 1 if out_dt == BF16 else 3, out_dt))


@pytest.mark.parametrize("rows,cols", [(200, 300), (300, 200)])
def test_schedules(rows, cols):
    g = gradients(1, rows, cols)
    for steps in (1, 2, 9):
        x, o = orthogonalize(g, FP32, FP32, 3, steps=steps)
        # nine steps pass on nine steps' errors
        check(o, plain(x, steps), 2 * tolerance(rows, cols, 3, FP32))
    cubic = [(1.5, -0.5, 0.0)] * 12
    x, o = orthogonalize(g, FP32, FP32, 3, coefs=cubic)
    check(o, plain(x, coefs=cubic), 3 * tolerance(rows, cols, 3, FP32))
    mixed = [(4.0, -6.0, 3.0), (3.4445, -4.7750, 2.0315), (2.0, -1.5, 0.5)]
    x, o = orthogonalize(g, FP32, FP32, 3, coefs=mixed)
    check(o, plain(x, coefs=mixed), tolerance(rows, cols, 3, FP32))


def test_scale_of_the_input_does_not_matter():
    # but for eps, 1e-7 against a norm of 2e-4 at the first
    g = gradients(1, 150, 170)
    for s in (1e-4, 1.0, 1e10, 1e25):      # |g|^2 passes fp32's range at the last
        x, o = orthogonalize(g * s, FP32, FP32, 3)
        check(o, plain(x), tolerance(150, 170, 3, FP32) + 1e-5)


def test_zeros_give_zeros_and_non_finite_values_stay_in_their_matrix():
    g = gradients(4, 140, 200)
    g[0] = 0
    g[1, 3, 5] = float("nan")
    g[2, 139, 199] = float("inf")
    x, o = orthogonalize(g, FP32, BF16)
    assert bool((o[0] == 0).all())
    assert bool(torch.isnan(o[1]).all()) and bool(torch.isnan(o[2]).all())
    check(o[3:], plain(x[3:]), tolerance(140, 200, 1, BF16))


@pytest.mark.parametrize("rows,cols", [(1, 4), (60, 80)])
def test_a_single_entry(rows, cols):
    # rank one: the singular value 1 goes where the scalar iteration takes it
    g = torch.zeros(1, rows, cols, device="cuda")
    g[0, 0, cols - 1] = -3.0
    x, o = orthogonalize(g, FP32, FP32, 3)
    check(o, plain(x), tolerance(rows, cols, 3, FP32))


def test_in_place_same_bits_other_stream_and_graph():
    g = gradients(3, 260, 390).to(torch.bfloat16)
    d = z.matrices(260, 390, batch=3, dtype=BF16)
    ws = torch.empty(z.zero_orthogonalize_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(g)
    z.zero_orthogonalize(d, g, out, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    again = torch.zeros_like(out)
    z.zero_orthogonalize(d, g, again, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, again)
    graph = torch.cuda.CUDAGraph()
    again.zero_()
    with torch.cuda.graph(graph):
        z.zero_orthogonalize(d, g, again, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    z.zero_orthogonalize(d, g, g, ws)             # over its own input
    assert torch.equal(out, g)


@pytest.mark.parametrize("rows,cols", [(40, 64), (260, 384)])
def test_results_beside_their_inputs_in_one_buffer(rows, cols):
    buf = torch.zeros(3, rows, 2 * cols, device="cuda", dtype=torch.bfloat16)
    g = gradients(3, rows, cols).to(torch.bfloat16)
    buf[:, :, :cols] = g
    packed = z.matrices(rows, cols, batch=3, dtype=BF16)
    d = z.matrices(rows, cols, batch=3, dtype=BF16, in_ld=2 * cols, out_ld=2 * cols)
    ws = torch.empty(z.zero_orthogonalize_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    want = torch.empty_like(g)
    z.zero_orthogonalize(packed, g, want, ws)
    z.zero_orthogonalize(d, buf, buf[:, :, cols:], ws)
    assert torch.equal(buf[:, :, cols:], want) and torch.equal(buf[:, :, :cols], g)


# ------------------------------------------------------------------ Muon step
class Job:
    def __init__(self, rows, cols, batch=1, n_d=2, dt=BF16, pdt=None, gap=0, seed=0, **hp):
        self.rows, self.cols, self.batch, self.n_d, self.dt = rows, cols, batch, n_d, dt
        self.pdt = dt if pdt is None else pdt
        self.stride = (rows * cols + 7) // 8 * 8 + gap
        self.size = batch * self.stride + 8
        self.seed = seed
        self.hp = dict(dict(lr=0.02, momentum=0.95, weight_decay=0.1, rms_scale=0.2, nesterov=True, loss_scale=1.0), **hp)
        self.desc = z.matrices(rows, cols, batch=batch, dtype=dt, out_dtype=self.pdt, stride=self.stride)
        nan = lambda t: torch.full((self.size,), float("nan"), dtype=t, device="cuda")  # noqa: E731
        self.momentum, self.master, self.lp = nan(torch.float32), nan(torch.float32), nan(TORCH[self.pdt])
        self.grads = [nan(TORCH[dt]) for _ in range(n_d)]
        self.view(self.momentum).copy_(gradients(batch, rows, cols, seed + 1) * 3)
        self.view(self.master).copy_(2 * gradients(batch, rows, cols, seed + 2))
        self.ws = torch.full((z.zero_muon_workspace_bytes(self.desc),), 0xFF, dtype=torch.uint8, device="cuda")
        self.sc = torch.zeros(256, dtype=torch.uint8, device="cuda")
        z.zero_scalars_init(self.sc)

    def view(self, t):
        return torch.as_strided(t, (self.batch, self.rows, self.cols), (self.stride, self.cols, 1))

    def new_grads(self, step):
        for q, t in enumerate(self.grads):
            self.view(t).copy_((self.hp["loss_scale"] * gradients(self.batch, self.rows, self.cols, 100 * step + q + 50)).to(t.dtype))

    def step_and_check(self, stream=None):
        hp = z.muon_hparams(**self.hp)
        m0, w0 = self.view(self.momentum).double(), self.view(self.master).double()
        # the mean as the step states it: fp32, rank order
        acc = torch.zeros(self.batch, self.rows, self.cols, device="cuda")
        for t in self.grads:
            acc = acc + self.view(t).float()
        mean = acc / (self.n_d * self.hp["loss_scale"])
        z.zero_muon_step(self.desc, hp, self.grads, self.momentum, self.master, self.lp, self.ws, self.sc, stream=stream)
        torch.cuda.synchronize()
        assert z.read_scalars(self.sc).status == 0
        mu = self.hp["momentum"]
        m = mu * m0 + mean.double()
        got_m = self.view(self.momentum).double()
        u32 = 2.0 ** -24
        # mu is 0.95 rounded to fp32, one product, one sum
        assert bool(((got_m - m).abs() <= 3 * u32 * (m0.abs() + mean.double().abs())).all())
        u = mean.double() + mu * m if self.hp["nesterov"] else m
        r, c = self.rows, self.cols
        scale = self.hp["rms_scale"] * max(r, c) ** 0.5 if self.hp["rms_scale"] > 0 else max(1.0, r / c) ** 0.5
        step = self.hp["lr"] * scale
        o = plain(u)
        w = w0 * (1 - self.hp["lr"] * self.hp["weight_decay"]) - step * o
        got_w = self.view(self.master).double()
        tol = tolerance(r, c, 3, FP32) + 1e-6       # u's own roundings in fp32, passed on
        err = (got_w - w)
        for i in range(self.batch):
            rounding = 4 * u32 * (w0[i].abs() + step * o[i].abs())
            assert float((err[i].abs() - rounding).clamp(min=0).norm()) <= step * tol * float(o[i].norm())
            assert bool((err[i].abs() <= rounding + 8 * step * tol * o[i].abs().max()).all())
        assert torch.equal(self.view(self.lp), self.view(self.master).to(TORCH[self.pdt]))
        for t in (self.momentum, self.master, self.lp):
            k = t.clone()
            self.view(k).fill_(float("nan"))
            assert bool(torch.isnan(k).all())


@pytest.mark.parametrize("rows,cols,batch,n_d,dt,kw", [
    (1, 1, 1, 1, BF16, {}), (1, 40, 1, 3, FP16, {}), (33, 17, 2, 2, BF16, {}), (64, 64, 1, 8, BF16, {}),
    (129, 300, 3, 5, FP16, {}), (300, 129, 2, 4, BF16, dict(gap=16)), (768, 768, 1, 8, BF16, {}),
    (100, 60, 40, 2, BF16, dict(rms_scale=0.0)), (200, 256, 1, 16, BF16, dict(nesterov=False)),
    (96, 160, 1, 4, FP16, dict(loss_scale=1024.0)), (160, 96, 1, 2, BF16, dict(momentum=0.0, weight_decay=0.0)),
    (77, 131, 1, 4, BF16, dict(pdt=FP16)), (80, 80, 1, 256, BF16, {})])
def test_muon_step(rows, cols, batch, n_d, dt, kw):
    job = Job(rows, cols, batch, n_d, dt, **kw)
    for step in range(2):
        job.new_grads(step)
        job.step_and_check()


def test_muon_without_weights_out_and_on_another_stream():
    job = Job(130, 140)
    job.new_grads(0)
    torch.cuda.synchronize()
    job.step_and_check(stream=torch.cuda.Stream())
    before = job.lp.clone()
    z.zero_muon_step(job.desc, z.muon_hparams(**job.hp), job.grads, job.momentum, job.master, None, job.ws)
    torch.cuda.synchronize()
    assert torch.equal(before.view(torch.int16), job.lp.view(torch.int16))


def test_zero_gradients_and_momentum_only_decay_the_weights():
    job = Job(50, 70, nesterov=True)
    for t in job.grads:
        job.view(t).zero_()
    job.view(job.momentum).zero_()
    w0 = job.view(job.master).clone()
    job.step_and_check()
    decay = np.float32(1.0 - float(np.float32(0.02)) * float(np.float32(0.1)))
    assert torch.equal(job.view(job.master), w0 * float(decay))


# -------------------------------------------------------------- bounded waits
def test_matrix_product_timeout_reports_and_context_survives():
    sc = torch.zeros(256, dtype=torch.uint8, device="cuda")
    scratch = torch.zeros(16384, dtype=torch.uint8, device="cuda")
    z.zero_scalars_init(sc)
    z.zero_debug_matmul_timeout(scratch, sc, 2_000_000)
    assert z.read_scalars(sc).status & z.ZERO_DEV_TIMEOUT
    assert torch.count_nonzero(scratch).item() == 0
    g = gradients(1, 100, 100)
    x, o = orthogonalize(g, FP32, FP32, 3)
    check(o, plain(x), tolerance(100, 100, 3, FP32))
