"""The norms' gradient of no rows, and what calls without y or without w_pre hand back."""
import pytest
import torch

from activation_sparse_transformer_amd import twell

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_no_rows_beside_weights_that_are_no_numbers(bad):
    """A sum over no rows is zero, whatever it would be multiplied by."""
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    odd = torch.full((64,), bad, device="cuda")
    for post, gate in ((odd, w), (w, odd), (odd, odd)):
        full = lambda: torch.full((64,), 7.0, device="cuda")
        got = twell.twell_norm_backward(e, e, e, e, w_post=post, gate=gate, w_pre=odd,
                                        out=twell.NormGrads(e, e, full(), full(), full()))
        for t in (got.dw_post, got.dgate, got.dw_pre):
            assert torch.equal(t, torch.zeros(64, device="cuda"))
