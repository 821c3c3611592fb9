"""Layer norm on the GPU against a plain evaluation in 64 bits.

Tolerances, element by element, from the arithmetic: each result is rounded
once to its type (unit roundoff U, and half the smallest subnormal for fp16);
before that, fp32 sums whose longest chain of additions is D deep are off by
at most D * 2^-24 of the sum of the terms' magnitudes, and each further fp32
operation by 2^-24 of its result."""
import numpy as np
import pytest
import torch

import zero_optimizer_step_02_gb300 as z

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = z.ZERO_BF16, z.ZERO_FP16, z.ZERO_FP32
TORCH = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32}
UNIT = {BF16: 2.0 ** -8, FP16: 2.0 ** -11, FP32: 2.0 ** -24}
TINY = {BF16: 0.0, FP16: 2.0 ** -25, FP32: 0.0}
U32 = 2.0 ** -24
EPS = 1e-5


def f64(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Inputs of one layer norm; pad: extra columns between rows; shift: the
    first element's offset into its buffer (in elements)."""

    def __init__(self, rows, cols, dt=BF16, wdt=FP32, pad=0, shift=0, seed=0, gain=True, bias=True, offset=0.0,
                 scale=1.0):
        g = torch.Generator().manual_seed(1000 * rows + cols + seed)
        self.rows, self.cols, self.dt, self.wdt = rows, cols, dt, wdt
        self.stride = cols + pad
        self.shift = shift
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.x = self.place(rnd(rows, cols) * scale * torch.exp(0.3 * rnd(cols)) + offset)
        self.dy = self.place(0.1 * rnd(rows, cols))
        self.y = self.place(torch.full((rows, cols), 7.0))
        self.dx = self.place(torch.full((rows, cols), 7.0))
        w = lambda t: torch.cat([torch.zeros(shift), t]).to(TORCH[wdt]).cuda()[shift:]  # noqa: E731
        self.gain = w(1.0 + 0.2 * rnd(cols)) if gain else None
        self.bias = w(0.2 * rnd(cols)) if bias else None
        self.dgain, self.dbias = w(torch.full((cols,), 7.0)), w(torch.full((cols,), 7.0))
        self.mean, self.rstd = torch.full((rows,), 7.0).cuda(), torch.full((rows,), 7.0).cuda()
        s = self.stride
        self.desc = z.layernorm(rows, cols, dtype=dt, w_dtype=wdt, eps=EPS, x_stride=s, y_stride=s, dy_stride=s,
                                dx_stride=s)
        self.ws = torch.full((z.zero_layernorm_workspace_bytes(self.desc),), 0xFF, dtype=torch.uint8, device="cuda")

    def place(self, t):
        """t inside a guarded wider buffer of NaN (what lies around must be neither read into results nor written)."""
        buf = torch.full((self.shift + max(self.rows, 1) * self.stride + 16,), float("nan"), dtype=TORCH[self.dt])
        v = buf[self.shift: self.shift + max(self.rows, 1) * self.stride].view(max(self.rows, 1), self.stride)
        v[: self.rows, : self.cols] = t.to(TORCH[self.dt])
        buf = buf.cuda()
        out = buf[self.shift: self.shift + max(self.rows, 1) * self.stride].view(-1, self.stride)[: self.rows, : self.cols]
        self.buffers = getattr(self, "buffers", []) + [(buf, out)]
        return out

    def guards_intact(self):
        for buf, out in self.buffers:
            c = buf.clone()
            c[self.shift: self.shift + max(self.rows, 1) * self.stride].view(-1, self.stride)[: self.rows, : self.cols] = float("nan")
            assert bool(torch.isnan(c).all())

    def forward(self):
        z.zero_layernorm_forward(self.desc, self.x, self.gain, self.bias, self.y, self.mean, self.rstd)

    def backward(self, **kw):
        a = dict(dx=self.dx, dgain=self.dgain, dbias=self.dbias)
        a.update(kw)
        z.zero_layernorm_backward(self.desc, self.dy, self.x, self.gain, self.mean, self.rstd, a["dx"], a["dgain"],
                                  a["dbias"], self.ws)

    # ------------------------------------------------ plain evaluation, 64 bits
    def weights64(self):
        g = np.ones(self.cols) if self.gain is None else f64(self.gain)
        b = np.zeros(self.cols) if self.bias is None else f64(self.bias)
        return g, b

    def check_forward(self):
        x = f64(self.x)
        g, b = self.weights64()
        mean = x.mean(1, keepdims=True)
        var = ((x - mean) ** 2).mean(1, keepdims=True)
        rstd = 1.0 / np.sqrt(var + EPS)
        y = (x - mean) * rstd * g + b
        depth = 16 + self.cols / 32
        # a mean off by e shifts xhat by e*rstd; rstd is off by half the relative error of its sum of squares
        e_mean = depth * U32 * np.abs(x).mean(1, keepdims=True) + U32 * np.abs(mean)
        e_rstd = rstd * (depth * U32 + 4 * U32) + rstd ** 3 * e_mean ** 2
        e_y = np.abs(g) * (e_mean * rstd + 2 * U32 * np.abs(x) * rstd + np.abs(x - mean) * e_rstd) + 4 * U32 * (np.abs((x - mean) * rstd * g) + np.abs(b))
        assert np.all(np.abs(f64(self.mean) - mean[:, 0]) <= e_mean[:, 0])
        assert np.all(np.abs(f64(self.rstd) - rstd[:, 0]) <= e_rstd[:, 0])
        got = f64(self.y)
        assert np.all(np.abs(got - y) <= UNIT[self.dt] * (np.abs(y) + e_y) + e_y + TINY[self.dt])

    def check_backward(self, dx=None, dgain=True, dbias=True):
        x, dy = f64(self.x), f64(self.dy)
        g, _ = self.weights64()
        mean, rstd = f64(self.mean)[:, None], f64(self.rstd)[:, None]
        xhat = (x - mean) * rstd
        e_x = 3 * U32 * (np.abs(x) + np.abs(mean)) * rstd
        h = dy * g
        m1, m2 = h.mean(1, keepdims=True), (h * xhat).mean(1, keepdims=True)
        want = rstd * (h - m1 - xhat * m2)
        depth = 16 + self.cols / 32
        e1 = (depth + 2) * U32 * np.abs(h).mean(1, keepdims=True)
        e2 = (depth + 4) * U32 * np.abs(h * xhat).mean(1, keepdims=True) + (np.abs(h) * e_x).mean(1, keepdims=True)
        e = rstd * (4 * U32 * (np.abs(h) + np.abs(m1) + np.abs(xhat * m2)) + e1 + np.abs(xhat) * e2 + e_x * np.abs(m2))
        got = f64(self.dx if dx is None else dx)
        assert np.all(np.abs(got - want) <= UNIT[self.dt] * (np.abs(want) + e) + e + TINY[self.dt])
        # columns: at most rows/32 + 16 additions in a chain
        depth = 16 + self.rows / 32
        for on, t, terms, e_t in ((dgain, self.dgain, dy * xhat, np.abs(dy) * e_x), (dbias, self.dbias, dy, 0 * dy)):
            if not on:
                continue
            w = terms.sum(0)
            e = (depth + 2) * U32 * np.abs(terms).sum(0) + e_t.sum(0)
            assert np.all(np.abs(f64(t) - w) <= UNIT[self.wdt] * (np.abs(w) + e) + e + TINY[self.wdt])


SHAPES = [(1, 1), (1, 17), (3, 33), (5, 8), (2, 256), (8, 768), (257, 768), (64, 1601), (31, 1024), (40, 1280),
          (7, 4096), (9, 2048), (700, 4096), (33, 8192), (3, 16384), (2, 16385), (3, 40000), (4100, 40), (1000, 72)]


@pytest.mark.parametrize("dt,wdt", [(BF16, FP32), (FP16, BF16), (FP32, FP32), (BF16, FP16), (FP32, BF16)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_and_backward(rows, cols, dt, wdt):
    c = Case(rows, cols, dt, wdt)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    c.guards_intact()


@pytest.mark.parametrize("pad,shift", [(1, 0), (0, 1), (8, 0), (5, 3), (8, 8)])
@pytest.mark.parametrize("rows,cols", [(13, 768), (6, 1601), (5, 4096), (4, 20000)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_strided_and_unaligned_views(rows, cols, dt, pad, shift):
    c = Case(rows, cols, dt, BF16, pad=pad, shift=shift)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    c.guards_intact()


@pytest.mark.parametrize("rows,cols", [(5000, 33), (5001, 130), (4000, 255), (3001, 511), (2500, 1023), (3000, 2047),
                                       (1300, 4095), (700, 5000), (400, 8191)])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_many_rows(rows, cols, dt):
    # full CTAs: as many row groups as registers and shared memory allow
    c = Case(rows, cols, dt, FP32)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    c.guards_intact()


@pytest.mark.parametrize("gain,bias", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("cols", [768, 1601, 8192])
def test_without_gain_or_bias(cols, gain, bias):
    c = Case(19, cols, gain=gain, bias=bias)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("cols", [96, 1601, 4096, 20000])
def test_missing_outputs_and_in_place(cols):
    c = Case(11, cols)
    c.forward()
    y = c.y.clone()
    z.zero_layernorm_forward(c.desc, c.x, c.gain, c.bias, c.y)           # no statistics stored
    assert torch.equal(y, c.y)
    for dg, db in ((None, c.dbias), (c.dgain, None), (None, None)):
        c.dgain.fill_(7.0)
        c.dbias.fill_(7.0)
        c.backward(dgain=dg, dbias=db)
        c.check_backward(dgain=dg is not None, dbias=db is not None)
        assert dg is not None or bool((c.dgain == 7.0).all())
        assert db is not None or bool((c.dbias == 7.0).all())
    c.backward()
    want = c.dx.clone()
    dy = c.dy.clone()
    c.backward(dx=c.dy)                                                  # dx over dy
    assert torch.equal(c.dy, want)
    c.dy.copy_(dy)
    x = c.x.clone()
    c.backward(dx=c.x)                                                   # dx over x
    assert torch.equal(c.x, want)
    c.x.copy_(x)
    z.zero_layernorm_forward(c.desc, c.x, c.gain, c.bias, c.x)           # y over x
    assert torch.equal(c.x, y)


@pytest.mark.parametrize("cols", [768, 1601])
def test_no_rows(cols):
    c = Case(0, cols)
    c.forward()
    c.backward()
    assert bool((c.dgain == 0).all()) and bool((c.dbias == 0).all())
    c.guards_intact()


@pytest.mark.parametrize("cols", [1, 40, 1601, 4096])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_constant_rows_give_the_bias(cols, dt):
    # the variance is zero: xhat is 0 up to the rounding of the mean (its
    # depth * 2^-24 relative error, times rstd = eps^-1/2)
    c = Case(4, cols, dt)
    c.x.fill_(0.5)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("cols", [768, 1601, 4096, 20000])
def test_large_offset_keeps_its_digits(cols):
    c = Case(6, cols, FP32, FP32, offset=1000.0)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()


@pytest.mark.parametrize("cols", [768, 1601, 4096])
def test_non_finite_rows_stay_in_their_rows(cols):
    c = Case(9, cols)
    c.x[2, 5] = float("inf")
    c.x[7, 0] = float("nan")
    c.forward()
    bad = [2, 7]
    good = [r for r in range(9) if r not in bad]
    assert bool(torch.isnan(c.y[bad]).all())
    assert bool(torch.isfinite(c.y[good].float()).all())
    d = Case(9, cols)
    d.forward()
    assert torch.equal(c.y[good], d.y[good])
    c.backward()
    d.backward()
    assert torch.equal(c.dx[good], d.dx[good]) and bool(torch.isnan(c.dx[bad]).all())
    assert bool(torch.isnan(c.dgain).all())                      # the bad rows belong to every column's sum
    assert torch.equal(c.dbias, d.dbias)                         # and dy has none


@pytest.mark.parametrize("rows,cols,dt", [(300, 768, BF16), (41, 1601, FP16), (2000, 4096, BF16)])
def test_same_bits_every_time_and_on_another_stream(rows, cols, dt):
    c = Case(rows, cols, dt, BF16)
    c.forward()
    c.backward()
    first = [t.clone() for t in (c.y, c.dx, c.dgain, c.dbias)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    z.zero_layernorm_forward(c.desc, c.x, c.gain, c.bias, c.y, c.mean, c.rstd, stream=s)
    z.zero_layernorm_backward(c.desc, c.dy, c.x, c.gain, c.mean, c.rstd, c.dx, c.dgain, c.dbias, c.ws, stream=s)
    s.synchronize()
    for a, b in zip(first, (c.y, c.dx, c.dgain, c.dbias)):
        assert torch.equal(a, b)


def _plain_forward(x, g, b):
    m = x.mean(1, keepdims=True)
    return (x - m) / np.sqrt(((x - m) ** 2).mean(1, keepdims=True) + EPS) * g + b


@pytest.mark.parametrize("rows,cols", [(5, 48), (9, 97), (3, 1024)])
def test_gradients_against_differences(rows, cols):
    # the derivative of sum(dy * y) along random directions, by central
    # differences of the 64-bit forward: with step h its own error is about
    # h^2 (third derivatives of order one here) plus 1e-16 / h
    c = Case(rows, cols, FP32, FP32)
    c.forward()
    c.backward()
    x, dy, g, b = f64(c.x), f64(c.dy), f64(c.gain), f64(c.bias)
    rng = np.random.default_rng(3)
    h = 1e-5
    for _ in range(4):
        vx, vg, vb = rng.standard_normal(x.shape), rng.standard_normal(cols), rng.standard_normal(cols)
        loss = lambda s: np.sum(dy * _plain_forward(x + s * vx, g + s * vg, b + s * vb))  # noqa: E731,B023
        diff = (loss(h) - loss(-h)) / (2 * h)
        got = np.sum(f64(c.dx) * vx) + np.sum(f64(c.dgain) * vg) + np.sum(f64(c.dbias) * vb)
        size = np.sum(np.abs(f64(c.dx) * vx)) + np.sum(np.abs(f64(c.dgain) * vg)) + np.sum(np.abs(f64(c.dbias) * vb))
        assert abs(got - diff) <= (16 + cols / 32 + 16) * U32 * size + 1e-8 * size


def test_graph_capture():
    c = Case(64, 768, BF16, BF16)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    want = [t.clone() for t in (c.y, c.dx, c.dgain, c.dbias)]
    for t in (c.y, c.dx, c.dgain, c.dbias):
        t.fill_(7.0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward()
        c.backward()
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, (c.y, c.dx, c.dgain, c.dbias)):
        assert torch.equal(a, b)


class Unlike(Case):
    """The same with arrays that lie differently: (pad, shift) of x, dy, y and dx."""

    def __init__(self, rows, cols, dt, lies, **kw):
        self.lies = iter(lies)
        super().__init__(rows, cols, dt, FP32, **kw)
        self.desc = z.layernorm(rows, cols, dtype=dt, w_dtype=FP32, eps=EPS, x_stride=self.x.stride(0),
                                dy_stride=self.dy.stride(0), y_stride=self.y.stride(0), dx_stride=self.dx.stride(0))

    def place(self, t):
        pad, shift = next(self.lies)
        buf = torch.full((shift + self.rows * (self.cols + pad) + 16,), float("nan"), dtype=TORCH[self.dt])
        buf[shift: shift + self.rows * (self.cols + pad)].view(self.rows, -1)[:, : self.cols] = t.to(TORCH[self.dt])
        buf = buf.cuda()
        out = buf[shift: shift + self.rows * (self.cols + pad)].view(self.rows, -1)[:, : self.cols]
        self.buffers = getattr(self, "buffers", []) + [(buf, out)]
        return out

    def guards_intact(self):
        for buf, out in self.buffers:
            c = buf.clone()
            torch.as_strided(c, out.shape, out.stride(), out.storage_offset()).fill_(float("nan"))
            assert bool(torch.isnan(c).all())


@pytest.mark.parametrize("lies", [((0, 0), (3, 1), (1, 2), (5, 0)), ((1, 1), (0, 0), (2, 7), (3, 3)),
                                  ((8, 0), (0, 8), (0, 1), (16, 0)), ((5, 0), (0, 0), (0, 0), (0, 0))])
@pytest.mark.parametrize("rows,cols", [(13, 40), (1201, 97), (90, 130), (13, 768), (301, 1601), (6, 4096), (1300, 2047),
                                       (200, 8189), (5, 8192)])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_arrays_that_lie_differently(rows, cols, dt, lies):
    c = Unlike(rows, cols, dt, lies)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    c.guards_intact()
    # over x, whatever dy's alignment
    x = c.x.clone()
    d = z.layernorm(rows, cols, dtype=dt, w_dtype=FP32, eps=EPS, x_stride=c.x.stride(0), dy_stride=c.dy.stride(0),
                    dx_stride=c.x.stride(0))
    z.zero_layernorm_backward(d, c.dy, c.x, c.gain, c.mean, c.rstd, c.x, c.dgain, c.dbias, c.ws)
    dx, c.x = c.x, x
    c.check_backward(dx=dx)
    c.guards_intact()


# rows of which several share a warp: one lane group's rows may run out before another's
@pytest.mark.parametrize("rows,cols", [(1, 64), (2, 8), (3, 57), (17, 64), (77, 31), (1234, 128), (1235, 121), (999, 113),
                                       (4001, 9), (9000, 32), (2433, 58), (40003, 24)])
@pytest.mark.parametrize("pad,shift", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_narrow_rows(rows, cols, dt, pad, shift):
    c = Case(rows, cols, dt, FP32, pad=pad, shift=shift)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward()
    c.guards_intact()


@pytest.mark.parametrize("cols", [24, 64, 120])
def test_non_finite_narrow_rows_stay_in_their_rows(cols):
    c, d = Case(37, cols), Case(37, cols)
    bad = [0, 6, 18, 36]
    c.x[bad, 3] = float("nan")
    good = [r for r in range(37) if r not in bad]
    for k in (c, d):
        k.forward()
        k.backward()
    assert torch.equal(c.y[good], d.y[good]) and torch.equal(c.dx[good], d.dx[good])
    assert bool(torch.isnan(c.y[bad]).all()) and bool(torch.isnan(c.dx[bad]).all())
    assert torch.equal(c.dbias, d.dbias)
