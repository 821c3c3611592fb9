"""The binding's check of an embedding's ids: no GPU needed, no call here reaches a launch."""
import pytest
import torch

from test_capi_model_host import z  # noqa: F401


def test_ids_that_are_not_as_a_call_reads_them(z):  # noqa: F811
    batch, x = torch.zeros(4, 9, dtype=torch.int64), torch.zeros(32, 8)
    for ids in (batch[:, :-1], batch.t(), batch.flatten()[::2], torch.zeros(31, dtype=torch.int64)):
        d = z.embedding(32 if ids.numel() >= 31 else ids.numel(), 10, 8)
        with pytest.raises(ValueError):
            z.zero_embedding_forward(d, ids, x, x)
        with pytest.raises(ValueError):
            z.zero_embedding_backward(d, ids, x, x, x)


def test_ids_that_are(z):  # noqa: F811
    """More ids than tokens, an address, no tokens: as before."""
    batch = torch.zeros(4, 9, dtype=torch.int64)
    for tokens, ids in ((32, batch), (36, batch.view(-1)), (8, batch[1:, :].contiguous()), (9, batch[2]), (4, 4096), (0, None)):
        z._capi._check_ids(z.embedding(tokens, 10, 8), ids)
