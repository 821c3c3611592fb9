"""Argument checks of the training operators (layer norm, matrix updates): no GPU needed, no
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


def test_layernorm_extents_stay_in_64_bits(z):
    d = z.layernorm(1 << 40, 64, x_stride=1 << 40)
    assert z.zero_layernorm_workspace_bytes(d) == 0
    assert ln_forward(z, d) == INVALID and ln_backward(z, d) == INVALID
    assert z.zero_layernorm_workspace_bytes(z.layernorm(1 << 40, 64)) > 0


def test_layernorm_workspace_size(z):
    assert z.zero_layernorm_workspace_bytes(z.layernorm(0, 64)) >= 256
    one = z.zero_layernorm_workspace_bytes(z.layernorm(1, 64))
    many = z.zero_layernorm_workspace_bytes(z.layernorm(1 << 20, 64))
    assert one % 256 == 0 and many % 256 == 0
    # bounded partial sums, and two row means for each row
    assert many <= 256 + 304 * 2 * 64 * 4 + 256 + (1 << 20) * 8 + 256


# ------------------------------------------------ orthogonalised updates, Muon
def orthogonalize(z, d, g=A, out=B, ws=C, sc=D):
    return z._capi.raw_status("zero_orthogonalize", ctypes.byref(d) if d is not None else None, g, out, ws, sc, None)


def muon(z, d, hp=None, n_d=2, ranks=(A, B), momentum=C, master=D, lp=E, ws=F, sc=G):
    hp = z.muon_hparams() if hp is None else hp
    arr = (ctypes.c_void_p * len(ranks))(*ranks) if ranks is not None else None
    return z._capi.raw_status("zero_muon_step", ctypes.byref(d) if d is not None else None, ctypes.byref(hp), n_d, arr,
                              momentum, master, lp, ws, sc, None)


BOUNDS = 6


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), INVALID), (dict(cols=-1), INVALID), (dict(batch=0), INVALID), (dict(dtype=5), INVALID),
    (dict(out_dtype=-1), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(products=2), INVALID), (dict(steps=-1), INVALID), (dict(steps=33), INVALID), (dict(in_ld=63), INVALID),
    (dict(out_ld=1), INVALID), (dict(stride=100), INVALID), (dict(out_stride=1), INVALID),
    (dict(rows=65537), BOUNDS), (dict(cols=65537), BOUNDS), (dict(batch=65536), BOUNDS),
    (dict(rows=65536, cols=65536), BOUNDS), (dict(rows=32768, cols=32768, batch=65535), BOUNDS),
    (dict(coefs=[(float("nan"), 0.0, 0.0)]), INVALID), (dict(coefs=[(100.0, 0.0, 0.0)] * 2), INVALID),
    (dict(coefs=[(3.0, -40.0, 1.0)]), INVALID)])
def test_matrices_descriptor_is_checked(z, kw, status):
    d = z.matrices(**dict(dict(rows=32, cols=64), **kw))
    assert z.zero_orthogonalize_workspace_bytes(d) == 0 and z.zero_muon_workspace_bytes(d) == 0
    assert orthogonalize(z, d) == status and muon(z, d) == status
    assert orthogonalize(z, None) == INVALID and muon(z, None) == INVALID


def test_schedules_that_fit_are_accepted(z):
    for coefs in (None, [(1.5, -0.5, 0.0)] * 32, [(1.875, -1.25, 0.375)] * 10, [(4.0, -6.0, 3.0)], [(1.0, 0.0, 0.0)]):
        assert z.zero_orthogonalize_workspace_bytes(z.matrices(32, 64, coefs=coefs)) > 0
    with pytest.raises(ValueError):
        z.matrices(32, 64, coefs=[(1.0, 2.0)])


def test_matrices_pointers_are_checked(z):
    d = z.matrices(32, 64, dtype=z.ZERO_BF16, out_dtype=z.ZERO_FP32)
    for k in ("g", "out", "ws"):
        assert orthogonalize(z, d, **{k: None}) == INVALID
    assert orthogonalize(z, d, g=A + 1) == MISALIGNED and orthogonalize(z, d, out=B + 2) == MISALIGNED
    assert orthogonalize(z, d, ws=C + 16) == MISALIGNED and orthogonalize(z, d, sc=D + 16) == MISALIGNED
    n = z.zero_orthogonalize_workspace_bytes(d)
    assert orthogonalize(z, d, g=C + n - 2) == INVALID and orthogonalize(z, d, out=C - 4) == INVALID


def test_a_batch_lies_on_its_own_inputs_only(z):
    """The matrices of a batch are under way side by side: a result on another one's input is refused."""
    d = z.matrices(32, 64, batch=3, dtype=z.ZERO_BF16)
    assert orthogonalize(z, d, g=A, out=A + 32 * 64 * 2) == INVALID          # on the next one
    assert orthogonalize(z, d, g=A, out=A + 2) == INVALID
    for kw in (dict(out_dtype=z.ZERO_FP32), dict(out_ld=65), dict(out_stride=32 * 64 + 64)):
        assert orthogonalize(z, z.matrices(32, 64, batch=3, dtype=z.ZERO_BF16, **kw), g=A, out=A) == INVALID
    # columns cut from one wide buffer: 128 bytes apart is side by side, 126 is not
    wide = z.matrices(32, 64, batch=3, dtype=z.ZERO_BF16, in_ld=128, out_ld=128)
    assert orthogonalize(z, wide, g=A, out=A + 126) == INVALID
    assert orthogonalize(z, wide, g=A + 128, out=A + 2) == INVALID
    # rows that do not repeat with the matrices
    odd = z.matrices(32, 64, batch=3, dtype=z.ZERO_BF16, in_ld=128, out_ld=128, stride=32 * 128 + 8, out_stride=32 * 128 + 8)
    assert orthogonalize(z, odd, g=A, out=A + 128) == INVALID


def test_muon_arguments_are_checked(z):
    d = z.matrices(32, 64)
    for k in ("ranks", "momentum", "master", "ws"):
        assert muon(z, d, **{k: None}) == INVALID
    assert muon(z, d, ranks=(A, None)) == INVALID and muon(z, d, n_d=0) == INVALID and muon(z, d, n_d=257) == INVALID
    for k, v in (("ranks", (A, B + 2)), ("momentum", C + 4), ("master", D + 4), ("lp", E + 2), ("ws", F + 16), ("sc", G + 8)):
        assert muon(z, d, **{k: v}) == MISALIGNED
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(momentum=1.0), dict(momentum=-0.1), dict(weight_decay=-1.0),
               dict(rms_scale=float("inf")), dict(loss_scale=-2.0)):
        assert muon(z, d, hp=z.muon_hparams(**kw)) == INVALID
    for kw in (dict(dtype=z.ZERO_FP32), dict(out_dtype=z.ZERO_FP32), dict(in_ld=72), dict(out_ld=72),
               dict(out_stride=4096)):
        assert muon(z, z.matrices(32, 64, **kw)) == INVALID
    assert muon(z, z.matrices(5, 5, batch=2)) == MISALIGNED                 # 25 elements: the second matrix is unaligned
    size = 32 * 64
    assert muon(z, d, momentum=D + 4 * size - 16) == INVALID                # over the end of master
    assert muon(z, d, lp=C + 16) == INVALID and muon(z, d, master=A + 16) == INVALID
    assert muon(z, d, ws=B) == INVALID and muon(z, d, lp=B + 2 * size - 16) == INVALID


def test_matmul_timeout_arguments_are_checked(z):
    call = lambda *a: z._capi.raw_status("zero_debug_matmul_timeout", *a, None)  # noqa: E731
    assert call(None, A, 1000) == INVALID and call(A, None, 1000) == INVALID
    assert call(A + 16, B, 1000) == MISALIGNED and call(A, B + 16, 1000) == MISALIGNED
    assert call(A, B, 0) == INVALID and call(A, B, 10_000_000_001) == INVALID
