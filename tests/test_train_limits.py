"""Limits of the operators around the layer: sizes and scales at the ends of their ranges, in
calls that end in the host's checks."""
import ctypes

import pytest
import torch

from activation_sparse_transformer_amd import twell

P = 4096  # an aligned address that no call below reads
OK, BAD, UNSUPPORTED = twell.TWELL_OK, twell.TWELL_ERR_INVALID_ARG, twell.TWELL_ERR_UNSUPPORTED


@pytest.mark.parametrize("scale,code", [(2.0 ** 127, OK), (1e-45, OK), (1.8e38, BAD), (3.4e38, BAD)])
def test_logprob_scale(scale, code):
    """scale * log2(e) has to be a float32: the exponents are formed with it."""
    lib = twell.load()
    s = twell.LogprobShape(0, 64, 64, 0, 8, 0, scale, 0)
    assert lib.twell_logprob_forward(ctypes.byref(s), P, P, P, P, P, None, None, None, 0,
                                     None) == code
    assert lib.twell_logprob_backward(ctypes.byref(s), P, P, P, None, P, None, P, 64, None) == code


def test_act8_widths_at_the_end_of_int32():
    """Blocks and code rows are counted without overflow; a row of codes has to be under 2^31."""
    lib = twell.load()
    a = twell.Act8Struct(P, P)
    both = lambda n, d: {lib.twell_act8_pack(n, d, 1, P, ctypes.byref(a), None),
                         lib.twell_act8_unpack(n, d, 1, ctypes.byref(a), P, None)}
    top = 2 ** 31
    assert both(0, top - 16) == {OK}
    assert both(8, top - 16) == {UNSUPPORTED}   # 2^27 blocks
    assert both(0, top - 8) == both(1, top - 8) == {UNSUPPORTED}


def test_sizes_past_int32_are_refused():
    """The structures hold 32-bit sizes; a larger one must not be cut to its low bits."""
    big = 2 ** 32 + 128
    x = torch.empty((1, big), dtype=torch.bfloat16, device="meta")
    ids = torch.empty((1,), dtype=torch.int64, device="meta")
    for call in (lambda: twell.twell_act8_pack(x),
                 lambda: twell.twell_act8_unpack(twell.Act8.empty(1, big, torch.bfloat16, "meta")),
                 lambda: twell.twell_embed_forward(x, ids),
                 lambda: twell.twell_embed_backward(x, ids, 10),
                 lambda: twell.twell_embed_backward(x[:, :64].contiguous(), ids, big),
                 lambda: twell.embed_backward_workspace(1, 8, big, "meta"),
                 lambda: twell.twell_logprob_forward(x, ids),
                 lambda: twell.twell_logprob_forward(x[:, :64], ids, top=big),
                 lambda: twell.logprob_workspace(1, big, 0, torch.float32, "meta"),
                 lambda: twell.make_shape(1, big, 512, 64, 4, torch.float32)):
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_lookup_in_the_largest_tables():
    """Only the gradient's launches are bound by the table's size."""
    lib = twell.load()
    s = twell.EmbedShape(0, 1 << 20, 8192, 1, 8, 1.0, 0)  # 2^33 elements
    assert lib.twell_embed_forward(ctypes.byref(s), P, None, None, None) == OK
    assert lib.twell_embed_backward(ctypes.byref(s), None, None, P, P, 1 << 40, None) == UNSUPPORTED
    assert lib.twell_embed_backward_workspace_size(ctypes.byref(s)) == 0


def test_embedding_gradient_of_almost_2_31_tokens():
    """Its loops over one id's tokens step by up to 1024 past the last of them, in int32."""
    lib = twell.load()
    s = lambda n: ctypes.byref(twell.EmbedShape(n, 10, 8, 1, 8, 1.0, 0))
    size = lib.twell_embed_backward_workspace_size
    assert size(s(2 ** 31 - 1024)) > 0
    for n in (2 ** 31 - 1023, 2 ** 31 - 1):
        assert size(s(n)) == 0
        assert lib.twell_embed_backward(s(n), P, P, P, P, 1 << 40, None) == UNSUPPORTED
