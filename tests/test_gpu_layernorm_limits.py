"""Layer norm where it can go wrong beside its shapes: calls from two host
threads, rows of huge values, widths above 8192 with many rows."""
import ctypes
import threading

import numpy as np
import pytest
import torch

import zero_optimizer_step_02_gb300 as z
from test_gpu_layernorm import BF16, FP32, TORCH, U32, UNIT, Unlike, f64

pytestmark = pytest.mark.gpu


def test_two_host_threads_each_with_its_own_stream():
    # two widths of one kernel that ask for different amounts of shared memory;
    # the threads share no workspace, so no order between their calls is asked
    # for and each call has to succeed
    calls, errors = 3000, []
    start = threading.Barrier(2)

    def work(cols):
        x = torch.randn(2048, cols, device="cuda").bfloat16()
        dy = torch.randn(2048, cols, device="cuda").bfloat16()
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = torch.empty(2048, device="cuda"), torch.empty(2048, device="cuda")
        dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        d = z.layernorm(2048, cols)
        ws = torch.empty(z.zero_layernorm_workspace_bytes(d), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        ptr = [ctypes.c_void_p(t.data_ptr()) for t in (x, y, mean, rstd, dy, dx, dg, db, ws)]
        stream = ctypes.c_void_p(s.cuda_stream)
        start.wait()
        for _ in range(calls):
            a = z._capi.raw_status("zero_layernorm_forward", ctypes.byref(d), ptr[0], None, None, ptr[1], ptr[2], ptr[3],
                                   stream)
            b = z._capi.raw_status("zero_layernorm_backward", ctypes.byref(d), ptr[4], ptr[0], None, ptr[2], ptr[3],
                                   ptr[5], ptr[6], ptr[7], ptr[8], stream)
            if a != 0 or b != 0:
                errors.append((cols, a, b))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in (4096, 1536)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert errors == []


# how the arrays lie: on whole words, alike inside them, differently
LIES = [((0, 0),) * 4, ((3, 1),) * 4, ((0, 0), (3, 1), (1, 2), (5, 0))]


@pytest.mark.parametrize("lies", LIES)
@pytest.mark.parametrize("cols,value,eps", [(8, 2.0 ** 120, 1e-5), (16, 2.0 ** 120, 1e-5), (64, 2.0 ** 120, 1e-5),
                                            (128, 2.0 ** 120, 1e-5), (256, 2.0 ** 110, 1e-30), (1024, 2.0 ** 110, 1e-30),
                                            (8192, 2.0 ** 110, 1e-30), (16384, 2.0 ** 110, 1e-30)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_constant_rows_of_huge_values_give_the_bias(cols, value, eps, dt, lies):
    # mean * rstd is past fp32's range, the mean of 2^n equal values is exact and xhat is 0
    rows = 5
    c = Unlike(rows, cols, dt, lies)
    c.desc.eps = eps
    c.x[2] = value
    c.forward()
    assert torch.equal(c.y[2], c.bias.to(TORCH[dt]))
    assert bool(torch.isfinite(c.y.float()).all())
    c.backward()
    dy, h = f64(c.dy), f64(c.dy)[2] * f64(c.gain)
    rstd = f64(c.rstd)[2]
    want = rstd * (h - h.mean())
    # a sum of `cols` terms, a product, a difference and two roundings of each
    e = rstd * U32 * ((16 + cols / 32 + 2) * np.abs(h).mean() + 4 * (np.abs(h) + np.abs(h).mean()))
    assert np.all(np.abs(f64(c.dx)[2] - want) <= UNIT[dt] * (np.abs(want) + e) + e)
    assert bool(torch.isfinite(c.dx.float()).all()) and bool(torch.isfinite(c.dgain).all())
    want = dy.sum(0)
    assert np.all(np.abs(f64(c.dbias) - want) <= (16 + rows) * U32 * np.abs(dy).sum(0))
    c.guards_intact()


@pytest.mark.parametrize("lies", LIES)
@pytest.mark.parametrize("cols", [24, 97, 768, 1601, 4096, 8192, 16384])
def test_fp32_rows_with_an_offset_are_centred_before_they_are_scaled(cols, lies):
    # against the formula with the kernel's own mean and rstd: one rounding each
    # for x - mean, the two products and the sum, none of the size of mean * rstd
    c = Unlike(6, cols, FP32, lies, offset=3000.0)
    c.forward()
    xhat = (f64(c.x) - f64(c.mean)[:, None]) * f64(c.rstd)[:, None]
    g, b = c.weights64()
    e = 4 * U32 * np.abs(xhat * g) + 2 * U32 * np.abs(b)
    assert np.all(np.abs(f64(c.y) - (xhat * g + b)) <= e)
    c.backward()
    c.check_backward()
    # dx likewise: the row's two means from the same xhat
    h = f64(c.dy) * g
    m1, m2 = h.mean(1, keepdims=True), (h * xhat).mean(1, keepdims=True)
    rstd = f64(c.rstd)[:, None]
    want = rstd * (h - m1 - xhat * m2)
    depth = 16 + cols / 32
    e = rstd * U32 * ((depth + 2) * np.abs(h).mean(1, keepdims=True) + (depth + 6) * np.abs(xhat) * np.abs(h * xhat).mean(1, keepdims=True)
                      + 4 * (np.abs(h) + np.abs(m1) + np.abs(xhat * m2)))
    assert np.all(np.abs(f64(c.dx) - want) <= U32 * np.abs(want) + e)
    c.guards_intact()


# Widths above 8192 with many rows to a part: even and odd numbers of them, a
# last pair that is one row, parts without a last row.  A column's sum is a
# chain over a part's rows (16 parts at least), then over every sixteenth part
# (304 at most), then a tree of sixteen.
@pytest.mark.parametrize("lies", [((0, 0),) * 4, ((8, 8),) * 4, ((3, 1),) * 4, ((0, 0), (3, 1), (1, 2), (5, 0))])
@pytest.mark.parametrize("rows,cols", [(700, 16384), (333, 20001), (129, 40000), (67, 65536), (1300, 8200), (33, 131073)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_many_rows_above_8192_columns(rows, cols, dt, lies):
    c = Unlike(rows, cols, dt, lies)
    c.forward()
    c.check_forward()
    c.backward()
    c.check_backward(dgain=False, dbias=False)
    x, dy = f64(c.x), f64(c.dy)
    mean, rstd = f64(c.mean)[:, None], f64(c.rstd)[:, None]
    xhat, e_x = (x - mean) * rstd, 3 * U32 * (np.abs(x) + np.abs(mean)) * rstd
    depth = rows / 16 + 1 + 304 / 16 + 4
    for t, terms, e_t in ((c.dgain, dy * xhat, np.abs(dy) * e_x), (c.dbias, dy, 0 * dy)):
        e = (depth + 2) * U32 * np.abs(terms).sum(0) + e_t.sum(0)
        want = terms.sum(0)
        assert np.all(np.abs(f64(t) - want) <= U32 * np.abs(want) + e)
    c.guards_intact()


@pytest.mark.parametrize("cols", [40, 768, 1601, 16384])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_one_row_in_place_whatever_its_strides(cols, dt):
    c = Unlike(1, cols, dt, LIES[0])
    c.forward()
    c.backward()
    d = z.layernorm(1, cols, dtype=dt, x_stride=cols + 3, y_stride=5 * cols, dy_stride=cols, dx_stride=2 * cols)
    for over in ("x", "dy"):
        k = Unlike(1, cols, dt, LIES[0])
        z.zero_layernorm_backward(d, k.dy, k.x, k.gain, c.mean, c.rstd, getattr(k, over), k.dgain, k.dbias, k.ws)
        assert torch.equal(getattr(k, over), c.dx) and torch.equal(k.dgain, c.dgain)
        k.guards_intact()
    z.zero_layernorm_forward(d, c.x, c.gain, c.bias, c.x)
    assert torch.equal(c.x, c.y)
    c.guards_intact()
