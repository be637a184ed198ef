"""Workspace of the backward pass from an 8-bit checkpoint: it is there for low peak memory, so
it must not need much more than the plain backward does.  Per entry (a TwELL slot or a stored dense
element) the plain one holds 16 + 4 S bytes and a dz of the storage type, this one 12 + 4 + 4 + 4 S:
with S = 8 slices, 52 against 50 (bfloat16) and 52 (float32)."""
import ctypes

import pytest
import torch

from activation_sparse_transformer_amd import twell


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,dm,dff", [(4096, 2048, 8192), (16384, 8192, 32768)])
def test_near_the_plain_backwards(n, dm, dff, dtype):
    lib = twell.load()
    shape = twell.make_shape(n, dm, dff, 128, 4, dtype)
    for cap in (n // 16, n // 4, n // 2):
        size = lib.ffn_sparse_backward_act8_workspace_size(ctypes.byref(shape), cap)
        plain = lib.ffn_sparse_backward_workspace_size(ctypes.byref(shape), cap)
        assert 0 < size <= 1.05 * plain
