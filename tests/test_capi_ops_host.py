"""Argument checks of the training operators (layer norm): no GPU needed, no
call here reaches a launch."""
import ctypes

import pytest

INVALID, MISALIGNED = 1, 2
A, B, C, D, E, F, G = (0x100000000 * k for k in range(1, 8))   # far apart, never dereferenced


@pytest.fixture(scope="module")
def z():
    import __graft_entry__
    __graft_entry__.build()
    import zero_optimizer_step_02_gb300 as z
    return z


def ln_forward(z, d, x=A, gain=B, bias=C, y=D, mean=E, rstd=F):
    return z._capi.raw_status("zero_layernorm_forward", ctypes.byref(d) if d is not None else None, x, gain, bias, y,
                              mean, rstd, None)


def ln_backward(z, d, dy=A, x=B, gain=C, mean=D, rstd=E, dx=F, dgain=G, dbias=G + 0x1000000, ws=0x9900000000):
    return z._capi.raw_status("zero_layernorm_backward", ctypes.byref(d) if d is not None else None, dy, x, gain,
                              mean, rstd, dx, dgain, dbias, ws, None)


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(cols=0), dict(cols=(1 << 24) + 1), dict(dtype=3), dict(w_dtype=-1),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(x_stride=63),
                                dict(y_stride=1), dict(dy_stride=-64), dict(dx_stride=63)])
def test_layernorm_descriptor_is_checked(z, kw):
    d = z.layernorm(**dict(dict(rows=4, cols=64), **kw))
    assert z.zero_layernorm_workspace_bytes(d) == 0
    assert ln_forward(z, d) == INVALID and ln_backward(z, d) == INVALID
    assert ln_forward(z, None) == INVALID and ln_backward(z, None) == INVALID


def test_layernorm_pointers_are_checked(z):
    d = z.layernorm(4, 64, dtype=z.ZERO_BF16, w_dtype=z.ZERO_FP32)
    assert ln_forward(z, d, x=None) == INVALID and ln_forward(z, d, y=None) == INVALID
    assert ln_forward(z, d, x=A + 1) == MISALIGNED and ln_forward(z, d, y=D + 1) == MISALIGNED
    assert ln_forward(z, d, gain=B + 2) == MISALIGNED and ln_forward(z, d, bias=C + 1) == MISALIGNED
    assert ln_forward(z, d, mean=E + 2) == MISALIGNED and ln_forward(z, d, rstd=F + 1) == MISALIGNED
    for k in ("dy", "x", "mean", "rstd", "dx", "ws"):
        assert ln_backward(z, d, **{k: None}) == INVALID
    assert ln_backward(z, d, dy=A + 1) == MISALIGNED and ln_backward(z, d, dgain=G + 2) == MISALIGNED
    assert ln_backward(z, d, mean=D + 2) == MISALIGNED and ln_backward(z, d, ws=0x9900000010) == MISALIGNED


def test_layernorm_overlap_is_checked(z):
    d = z.layernorm(4, 64, dtype=z.ZERO_BF16)
    assert ln_forward(z, d, x=A, y=A + 128) == INVALID            # one row down
    assert ln_forward(z, d, x=A, y=A + 2) == INVALID
    w = z.layernorm(4, 64, dtype=z.ZERO_BF16, x_stride=128)
    assert ln_forward(z, w, x=A, y=A) == INVALID                  # the same start, other strides
    assert ln_backward(z, d, dx=A + 128) == INVALID and ln_backward(z, d, dx=B + 128) == INVALID
    assert ln_backward(z, d, dbias=G) == INVALID
    assert ln_backward(z, d, dbias=G + 4) == INVALID
    wide = z.layernorm(4, 64, dtype=z.ZERO_BF16, x_stride=128, y_stride=128)
    assert ln_forward(z, wide, x=A, y=A + 126) == INVALID         # the last column of x's half
    assert ln_forward(z, wide, x=A + 128, y=A + 2) == INVALID


def test_layernorm_workspace_size(z):
    assert z.zero_layernorm_workspace_bytes(z.layernorm(0, 64)) >= 256
    one = z.zero_layernorm_workspace_bytes(z.layernorm(1, 64))
    many = z.zero_layernorm_workspace_bytes(z.layernorm(1 << 20, 64))
    assert one % 256 == 0 and many % 256 == 0
    # bounded partial sums, and two row means for each row
    assert many <= 256 + 304 * 2 * 64 * 4 + 256 + (1 << 20) * 8 + 256
