"""What a residual join writes may lie on nothing else: no GPU needed, no call here reaches a launch."""
import pytest

from test_capi_model_host import INVALID, P, join_backward, join_forward, z  # noqa: F401

VECTORS = ("post_gain", "post_bias", "gate", "pre_gain")
GRADIENTS = ("dpost_gain", "dpost_bias", "dgate", "dpre_gain", "dpre_bias")
ROW, BYTES = 128, 512   # of [4, 64] 16-bit activations; vectors of 64 fp32 values are 256 bytes


def test_forward_results_on_vectors(z):  # noqa: F811
    d = z.residual_norm(4, 64)
    for out in ("hout", "y"):
        for v in VECTORS + ("pre_bias",):
            for at in (P[v], P[v] + 252, P[v] - BYTES + 16):
                assert join_forward(z, d, **{out: at}) == INVALID, (out, v)
    for v in VECTORS + ("pre_bias",):
        for at in (P[v], P[v] + 240, P[v] - 48):
            assert join_forward(z, d, stats=at) == INVALID, v


def test_backward_results_on_what_is_read(z):  # noqa: F811
    d = z.residual_norm(4, 64)
    t = z.residual_norm(4, 64, gate_stride=64)
    for out in ("dh", "do"):
        for at in (P["stats"], P["stats"] + 48, P["stats"] - BYTES + 16):
            assert join_backward(z, d, **{out: at}) == INVALID
        for v in VECTORS:
            for at in (P[v], P[v] + 252, P[v] - BYTES + 16):
                assert join_backward(z, d, **{out: at}) == INVALID, (out, v)
    assert join_backward(z, t, dgate=P["stats"] + 32) == INVALID and join_backward(z, t, dgate=P["post_bias"]) == INVALID
    for g in GRADIENTS:
        for at in (P["stats"], P["stats"] + 60, P["stats"] - 252):
            assert join_backward(z, d, **{g: at}) == INVALID, g
        for v in VECTORS:
            for at in (P[v], P[v] + 252, P[v] - 252):
                assert join_backward(z, d, **{g: at}) == INVALID, (g, v)


def test_workspace_on_vectors(z):  # noqa: F811
    d = z.residual_norm(4, 64)
    n = z.zero_residual_norm_workspace_bytes(d)
    for v in VECTORS:
        assert join_backward(z, d, ws=P[v]) == INVALID and join_backward(z, d, ws=P[v] - n + 256) == INVALID


@pytest.mark.parametrize("rows", [1, 4])
def test_vectors_beside_strided_rows(z, rows):  # noqa: F811
    """Rows 256 bytes apart, 128 of them a row's: what begins in a row's bytes, or reaches into the next row's, is refused.
    (What lies between the rows' bytes is not: such calls run, in the GPU tests.)"""
    d = z.residual_norm(rows, 64, stride=128, w_dtype=z.ZERO_BF16)   # vectors of 128 bytes
    for g in GRADIENTS:
        for on in ("dh", "do", "dy", "hout"):
            for at in (0, 126, -126) + ((256 + 64, 3 * 256 + 126, 2 * 256 - 2) if rows == 4 else ()):
                assert join_backward(z, d, **{g: P[on] + at}) == INVALID, (g, on, at)
    for out in ("dh", "do"):
        assert join_backward(z, d, **{out: P["pre_gain"] - 126}) == INVALID
