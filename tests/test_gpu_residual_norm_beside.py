"""What overlaps nothing is taken: statistics and gradients of vectors between the rows of the join's arrays, where no row has a
byte, give the same bits as apart; an array without an element has no place."""
import pytest
import torch

from test_gpu_residual_norm import VECTORS, Case, z  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gate", ["vector", "token"])
@pytest.mark.parametrize("pad", [64, 67])
def test_between_the_rows(z, gate, pad):  # noqa: F811
    rows, cols = 4, 64
    kw = dict(w="bf16", post="layer", pre="layer", gate=gate, pad=(pad,) * 4, seed=71)
    c, d = Case(z, rows, cols, "bf16", **kw), Case(z, rows, cols, "bf16", **kw)
    for k in VECTORS:
        if c.dw[k] is not None:
            c.dw[k] = torch.full((cols,), 7.0, device="cuda", dtype=torch.bfloat16)
    gap = lambda r, row: r.flat[row * r.ld + cols: (row + 1) * r.ld]  # noqa: E731
    for k, r in (("post_gain", d.dh), ("post_bias", d.do), ("gate", d.dy), ("pre_gain", d.hout), ("pre_bias", d.dhout)):
        if d.dw[k] is not None:
            d.dw[k] = gap(r, 1)[:cols]
    if pad == 64:   # on 16 bytes
        d.stats = gap(d.h, 2)[:32].view(torch.float32).view(rows, 4)
    for x in (c, d):
        x.forward()
        x.backward()
    torch.cuda.synchronize()
    assert torch.equal(c.stats[:rows], d.stats[:rows])
    for a, b in ((c.hout, d.hout), (c.y, d.y), (c.dh, d.dh), (c.do, d.do)) + (((c.dtok, d.dtok),) if gate == "token" else ()):
        assert torch.equal(a.v, b.v)
    for k in VECTORS:
        assert c.dw[k] is None or torch.equal(c.dw[k], d.dw[k])
    assert bool((gap(d.dh, 0) == 7.0).all()) and bool((gap(d.do, 2) == 7.0).all()) and bool((gap(d.dh, 1)[cols:] == 7.0).all())


def test_arrays_without_an_element(z):  # noqa: F811
    """Without rows, or tokens, an address says nothing, wherever it points."""
    c = Case(z, 0, 40, "bf16")
    w, dw, at = c.w, c.dw, c.ws.data_ptr() + 64
    z.zero_residual_norm_backward(c.desc, at, at, at, at, w["post_gain"], w["post_bias"], w["gate"], w["pre_gain"], at, at, at,
                                  dw["post_gain"], dw["post_bias"], dw["gate"], dw["pre_gain"], dw["pre_bias"], c.ws)
    for k in VECTORS:
        assert bool((dw[k][:40] == 0).all()) and bool((dw[k][40:] == 7.0).all())
    table = torch.full((10, 8), 7.0, device="cuda")
    d = z.embedding(0, 10, 8, dtype=z.ZERO_FP32, table_dtype=z.ZERO_FP32)
    ws = torch.empty(z.zero_embedding_workspace_bytes(d), dtype=torch.uint8, device="cuda")
    z.zero_embedding_backward(d, table.data_ptr() + 32, table.data_ptr() + 64, table, ws)
    assert bool((table == 0).all())
