"""The joins where a team takes more rows than its ring of stages holds (a row's slots are used again, sums take their buffers in
turn), in every form of the kernels; in place; beyond 2^31 elements."""
import pytest
import torch

from test_gpu_residual_norm import EPS, HALF, U, VECTORS, Case, both, kind, z, zt  # noqa: F401

pytestmark = pytest.mark.gpu
WHOLE, ALIKE, APART, SINGLE = ((0,) * 4, (0,) * 4), ((8,) * 4, (5,) * 4), ((3,) * 4, (1,) * 4), ((0, 1, 2, 3), (0,) * 4)


# Turns a team: rows over (teams in a CTA or cluster) x (152 SMs over the CTAs of a cluster) x (rows at a time); each more than
# the stages (two to four) and two.  Up to 2048 columns, up to 4096 (backward a row's norms share a barrier), above (clusters).
@pytest.mark.parametrize("rows,cols", [(9000, 768), (3000, 4096), (1500, 5000), (1100, 8192), (600, 16384)])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("gate", ["vector", "token"])
def test_whole_rows(z, rows, cols, dt, gate):  # noqa: F811
    both(z, rows, cols, dt, post="layer", pre="rms", gate=gate, seed=31)


@pytest.mark.parametrize("rows,cols", [(7000, 1601), (2500, 4001), (600, 9001)])
@pytest.mark.parametrize("pad,skew", [ALIKE, APART, SINGLE])
@pytest.mark.parametrize("dt", ["fp16", "fp32"])
@pytest.mark.parametrize("gate", ["vector", "token"])
def test_odd_rows(z, rows, cols, dt, gate, pad, skew):  # noqa: F811
    both(z, rows, cols, dt, post="rms", pre="layer", gate=gate, pad=pad, skew=skew, seed=32)


@pytest.mark.parametrize("rows,cols", [(20000, 40), (40000, 5)])
@pytest.mark.parametrize("pad,skew", [WHOLE, APART, SINGLE])
def test_teams_of_less_than_a_warp(z, rows, cols, pad, skew):  # noqa: F811
    both(z, rows, cols, "bf16", post="layer", pre="layer", pad=pad, skew=skew, seed=33)


@pytest.mark.parametrize("post,pre", [("none", "layer"), ("rms", "none"), ("none", "none"), ("layer", "layer")])
@pytest.mark.parametrize("rows,cols", [(1500, 4096), (600, 16384)])
def test_norms_left_out(z, post, pre, rows, cols):  # noqa: F811
    both(z, rows, cols, "bf16", post=post, pre=pre, seed=34)


@pytest.mark.parametrize("rows,cols", [(1500, 4096), (600, 16384)])
@pytest.mark.parametrize("pad,skew", [WHOLE, APART])
def test_in_place_with_a_gate_vector(z, rows, cols, pad, skew):  # noqa: F811
    """A row's do is stored a turn later than its dh: the same bits in place as apart."""
    kw = dict(post="layer", pre="rms", pad=pad, skew=skew, seed=35)
    c = both(z, rows, cols, "bf16", **kw)
    d = Case(z, rows, cols, "bf16", **kw)
    d.forward(hout=d.o.v, y=d.h.v)
    assert torch.equal(d.o.v, c.hout.v) and torch.equal(d.h.v, c.y.v)
    for dh_on, do_on in ((None, "dhout"), (None, "dy"), (None, "o"), (None, "hout"), ("dhout", "o"), ("dy", "dhout"), ("hout", "dy")):
        e = Case(z, rows, cols, "bf16", **kw)
        e.forward()
        to = {k: getattr(e, on).v for k, on in (("dh", dh_on), ("do", do_on)) if on}
        e.backward(**to)
        assert torch.equal(to.get("dh", e.dh.v), c.dh.v) and torch.equal(to.get("do", e.do.v), c.do.v), (dh_on, do_on)
        for k in VECTORS:
            assert torch.equal(c.dw[k], e.dw[k])


def test_more_elements_than_an_int_counts(z):  # noqa: F811
    """2.2e9 elements; rows from all over, the last ones too, against 64 bits."""
    rows, cols, dt = 530_001, 4096, torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(36)

    def array(size):
        x = torch.empty(rows, cols, dtype=dt, device="cuda")
        for at in range(0, rows, 100_000):
            x[at: at + 100_000].normal_(generator=g)
        return x.mul_(size)

    vec = lambda: 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")  # noqa: E731
    h, o, dy, dhout = array(2.0), array(1.0), array(0.125), array(0.125)
    hout, y, dh, do = (torch.empty_like(h) for _ in range(4))
    post_gain, gate, pre_gain = vec(), vec(), vec()
    stats = torch.empty(rows, 4, device="cuda")
    desc = z.residual_norm(rows, cols, post=kind(z, "rms"), pre=kind(z, "layer"), dtype=zt(z, dt), post_eps=EPS, pre_eps=EPS)
    ws = torch.empty(z.zero_residual_norm_workspace_bytes(desc), dtype=torch.uint8, device="cuda")
    z.zero_residual_norm_forward(desc, h, o, post_gain, None, gate, hout, pre_gain, None, y, stats)
    z.zero_residual_norm_backward(desc, dy, dhout, o, hout, post_gain, None, gate, pre_gain, stats, dh, do, None, None, None, None, None, ws)
    at = torch.cat([torch.arange(0, rows, 5003), torch.arange(rows - 9, rows), torch.arange(524_280, 524_297)]).cuda()
    f = lambda t: t[at].double()  # noqa: E731
    pg, gv, qg, x, ov = post_gain.double(), gate.double(), pre_gain.double(), f(hout), f(o)
    ro = 1 / torch.sqrt((ov * ov).mean(1, keepdim=True) + EPS)
    mean = x.mean(1, keepdim=True)
    rh = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + EPS)
    ohat, xhat = ov * ro, (x - mean) * rh
    # values of order one to ten: sums 32 deep and a few products, 2^-24 each, then one rounding of the result
    near = lambda got, want, size: bool(((f(got) - want).abs() <= HALF[dt] * 1.01 * want.abs() + 64 * U * size).all())  # noqa: E731
    assert near(hout, f(h) + gv * pg * ohat, f(h).abs() + (gv * pg * ohat).abs())
    assert near(y, qg * xhat, (qg * xhat).abs() + qg.abs())

    def through(u, xh, r, layer):
        got = u - xh * (u * xh).mean(1, keepdim=True) - (u.mean(1, keepdim=True) if layer else 0.0)
        return r * got, r * (u.abs() + xh.abs() * (u * xh).abs().mean(1, keepdim=True) + u.abs().mean(1, keepdim=True))

    d, d_size = through(f(dy) * qg, xhat, rh, True)
    d, d_size = d + f(dhout), d_size + f(dhout).abs()
    assert near(dh, d, d_size)
    want, size = through(d * gv * pg, ohat, ro, False)
    # d is off by up to 64 U of d_size already
    assert near(do, want, size + through(d_size * (gv * pg).abs(), ohat.abs(), ro, False)[1])
