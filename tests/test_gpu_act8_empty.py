"""The backward pass from a checkpoint of no rows, at a layer whose weight gradients are more
16-byte vectors than one launch has lanes: they are zeroed whole."""
import ctypes

import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import say


@pytest.mark.gpu
def test_no_rows_of_the_largest_layers():
    say("backward_act8 n=0, 2^20 x 16384")
    dm, dff = 16384, 1 << 20
    lib = twell.load()
    shape = twell.make_shape(0, dm, dff, 64, 4, torch.bfloat16)
    need = lib.ffn_sparse_backward_act8_workspace_size(ctypes.byref(shape), 0)
    ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
    # 64 GiB; both weight gradients are the same zeros
    dw = torch.empty((dff, dm), dtype=torch.float32, device="cuda").fill_(7)
    db = torch.full((dff,), 7.0, device="cuda")
    n_dense = torch.zeros((4,), dtype=torch.int32, device="cuda")
    h = twell.HybridStruct(None, None, None, None, None, n_dense.data_ptr(), 0)
    x8 = twell.Act8Struct(None, None)
    code = lib.ffn_sparse_backward_act8(
        ctypes.byref(shape), ctypes.byref(x8), None, None, ctypes.byref(h), None, None,
        dw.data_ptr(), db.data_ptr(), dw.data_ptr(), ws.data_ptr(), need,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert code == twell.TWELL_OK
    assert not db.any()
    for part in dw.view(-1).split(1 << 30):
        assert not part.any()
