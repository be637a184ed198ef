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
