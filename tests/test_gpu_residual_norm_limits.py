"""The join's backward pass on rows whose mean is large: normalised rows are those of the statistics given, (x - mean) * rstd."""
import pytest
import torch

from test_gpu_residual_norm import HALF, U, Case, z  # noqa: F401

pytestmark = pytest.mark.gpu
# whole words, alike inside them, rows of their own places
LIES = [((0, 0, 0, 0), (0, 0, 0, 0)), ((3, 3, 3, 3), (5, 5, 5, 5)), ((0, 1, 2, 3), (0, 0, 0, 0))]


def norm_gradient(u, xhat, rstd, cols, u_off):
    """rstd * (u - mean(u) - xhat * mean(u * xhat)) in 64 bits, and how far fp32 may be off: sums of `cols` terms, 16 + cols / 32 deep,
    a handful of products, x - mean and its product with rstd rounded once each; u itself is off by u_off."""
    mean = lambda t: t.mean(1, keepdim=True)  # noqa: E731
    want = rstd * (u - mean(u) - xhat * mean(u * xhat))
    a, x, deep = u.abs(), xhat.abs(), 16 + cols / 32
    off = rstd * U * ((deep + 2) * mean(a) + (deep + 6) * x * mean(a * x) + 4 * (a + mean(a) + x * mean(a * x)))
    return want, off + rstd * (u_off + mean(u_off) + x * mean(u_off * x))


def check(c):
    """The backward pass against the formula with the statistics that it was given."""
    f = lambda t: t.double()  # noqa: E731
    w, st, rows, cols = {k: f(v) for k, v in c.w.items() if v is not None}, f(c.stats[: c.rows]), c.rows, c.cols
    # a constant row's difference is 0 whatever the product (inf * 0 does not come up: both are finite)
    xhat, ohat = (f(c.hout.v) - st[:, 2:3]) * st[:, 3:4], (f(c.o.v) - st[:, 0:1]) * st[:, 1:2]
    dy, dhout, gate = f(c.dy.v), f(c.dhout.v), f(c.gate())
    u = dy * w["pre_gain"]
    d, d_off = norm_gradient(u, xhat, st[:, 3:4], cols, U * u.abs())
    d, d_off = d + dhout, d_off + U * (d.abs() + dhout.abs())
    p = ohat * w["post_gain"] + w["post_bias"]
    t = d * gate * w["post_gain"]
    t_off = (gate * w["post_gain"]).abs() * d_off + 4 * U * t.abs()
    do, do_off = norm_gradient(t, ohat, st[:, 1:2], cols, t_off)

    def near(got, want, off, dt):
        off = off + HALF[dt] * 1.01 * want.abs() + 1e-37
        far = (f(got) - want).abs()
        assert bool(torch.isfinite(got).all()) and bool((far <= off).all()), float((far / off).max())

    near(c.dh.v, c.res_scale * d, c.res_scale * d_off + U * d.abs(), c.dt)
    near(c.do.v, do, do_off, c.dt)
    deep = U * (rows + 32)
    p_off = 4 * U * ((ohat * w["post_gain"]).abs() + p.abs())
    dv, v_off = d * gate, gate.abs() * d_off + 2 * U * (d * gate).abs()
    sums = {"pre_gain": (dy * xhat, 4 * U * (dy * xhat).abs()), "pre_bias": (dy, 0 * dy), "post_gain": (dv * ohat, v_off * ohat.abs() + 4 * U * (dv * ohat).abs()),
            "post_bias": (dv, v_off)}
    if c.tok:
        near(c.dtok.v, d * p, d_off * p.abs() + d.abs() * p_off, c.dt)
    else:
        # gain * sum(d * ohat) + bias * sum(d): sizes of what is added up, not of the sum
        size = d.abs() * ((ohat * w["post_gain"]).abs() + w["post_bias"].abs())
        near(c.dw["gate"][:cols], (d * p).sum(0), (deep + 8 * U) * size.sum(0) + (d_off * size / d.abs().clamp(min=1e-300)).sum(0), c.wt)
    for k, (terms, off) in sums.items():
        near(c.dw[k][:cols], terms.sum(0), (deep + 8 * U) * terms.abs().sum(0) + off.sum(0), c.wt)
    for r in (c.dh, c.do):
        assert r.canaries()


@pytest.mark.parametrize("pad,skew", LIES)
@pytest.mark.parametrize("gate", ["vector", "token"])
@pytest.mark.parametrize("cols", [8, 200, 1601, 5000, 16384])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_constant_rows_of_huge_values(z, dt, cols, gate, pad, skew):  # noqa: F811
    """mean * rstd is past fp32's range; every x is the mean, and its normalised value 0."""
    c = Case(z, 6, cols, dt, post="layer", pre="layer", gate=gate, pad=pad, skew=skew, seed=22)
    c.forward()
    huge, rstd = 2.0 ** 120, 1e-5 ** -0.5
    c.o.v[2], c.hout.v[2], c.hout.v[4] = huge, -huge, huge
    c.stats[2] = torch.tensor([huge, rstd, -huge, rstd])
    c.stats[4, 2:] = torch.tensor([huge, rstd])
    c.backward()
    check(c)


@pytest.mark.parametrize("pad,skew", LIES)
@pytest.mark.parametrize("gate", ["vector", "token"])
@pytest.mark.parametrize("cols", [24, 97, 768, 1601, 4096, 8192, 16384])
def test_fp32_rows_with_an_offset(z, cols, gate, pad, skew):  # noqa: F811
    """None of the roundings is of the size of mean * rstd."""
    c = Case(z, 6, cols, "fp32", post="layer", pre="layer", gate=gate, pad=pad, skew=skew, seed=23, offset=3000.0)
    c.forward()
    c.backward()
    check(c)
