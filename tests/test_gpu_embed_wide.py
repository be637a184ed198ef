"""The token embedding at the widest row there is, 2^31 - 8 columns: column counts are rounded up
without leaving int32.  Values are small integers: equal exactly."""
import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import say


@pytest.mark.gpu
def test_widest_row():
    say("embed d_model 2^31 - 8")
    d = 2 ** 31 - 8
    ids = torch.tensor([0], device="cuda")
    at = [0, 1, 12345, d // 2, d - 9, d - 1]
    table = torch.ones((1, d), dtype=torch.bfloat16, device="cuda")
    table[0, at] = torch.arange(2.0, 8.0, device="cuda").bfloat16()
    out = torch.full_like(table, 9.0)
    twell.twell_embed_forward(table, ids, scale=2.0, out=out)
    assert out[0, at].tolist() == [4.0, 6.0, 8.0, 10.0, 12.0, 14.0]
    total = sum(float(p.sum(dtype=torch.float64)) for p in out[0].split(1 << 28))
    assert total == 2.0 * (d - 6) + 54.0
    del table
    grad = twell.twell_embed_backward(out, ids, 1, out=torch.full((1, d), 9.0, device="cuda"))
    assert all(torch.equal(g, o.float()) for g, o in zip(grad[0].split(1 << 28),
                                                         out[0].split(1 << 28)))


@pytest.mark.gpu
def test_lookup_in_a_table_past_2_33_elements():
    say("embed 2^20 + 1 ids of 8192")
    vocab, d = (1 << 20) + 1, 8192
    table = torch.empty((vocab, d), dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, vocab, 1 << 19, vocab - 2], device="cuda")
    for v, k in ((1.0, 0), (2.0, 1 << 19), (3.0, vocab - 2), (4.0, vocab - 1)):
        table[k] = v
    out = twell.twell_embed_forward(table, ids)
    want = torch.tensor([4.0, 1.0, 0.0, 2.0, 3.0], device="cuda").bfloat16()
    assert torch.equal(out, want[:, None].expand(5, d))
