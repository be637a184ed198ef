"""Widths of the backward pass from an 8-bit checkpoint: every multiple of 8 up to 16384 in both
dtypes, at those where its column slices differ in kind (one slice or eight, wholly covered by
their lanes or not, a shorter last one).

The layers hold small integers and every float32 sum is below 2^24 in magnitude, so results equal
the oracle's bit for bit; dx is rounded once."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from activation_sparse_transformer_amd import twell
from gpu_helpers import as_f32, as_f64, say
from oracle.train_oracle import act8_decode

DTYPES = [torch.bfloat16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_width_is_accepted(dtype):
    size = lambda d: twell.load().ffn_sparse_backward_act8_workspace_size(
        ctypes.byref(twell.make_shape(64, d, 512, 64, 8, dtype)), 64)
    assert [d for d in range(8, 16385, 8) if size(d) == 0] == []
    for d in (4, 60, 16392, 32768, 2 ** 31 - 8):
        assert size(d) == 0, d


def ternary(rng, shape, zero):
    a = rng.integers(-1, 2, size=shape).astype(np.float32)
    a[rng.random(shape) < zero] = 0
    return a


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("dm", [
    8, 1024, 1032, 1544, 2040, 2048,  # one slice of two vectors per lane, the second one partial
    2056, 2080, 4088, 4104,           # eight slices, the last one shorter
    4096,                             # eight of 512, covered wholly
    4128, 8200, 8256,
    16376, 16384,                     # the widest
])
def test_widths_integer_valued_exact(dm, dtype):
    say(f"backward_act8 width {dm} {dtype}")
    n, dff, T, C = 70, 192, 64, 8
    rng = np.random.default_rng(dm)
    wu, wd, dy = (ternary(rng, s, 0.6) for s in ((dff, dm), (dff, dm), (n, dm)))
    # every fourth row too full for its tiles, the others with a few units
    share = np.where(np.arange(n) % 4 == 0, 0.4, 0.03)[:, None]
    h = np.where(rng.random((n, dff)) < share, rng.integers(1, 4, size=(n, dff)), 0)
    x8 = twell.Act8.empty(n, dm, dtype, "cuda:0")
    x8.codes.zero_()
    x8.codes[:, :dm] = torch.from_numpy(ternary(rng, (n, dm), 0.5).astype(np.int8)).cuda()
    x8.scales.copy_(torch.from_numpy(
        rng.integers(1, 3, size=tuple(x8.scales.shape)).astype(np.float32)))
    to = lambda a: torch.from_numpy(a.astype(np.float32)).to(dtype).cuda()
    hy, status = twell.twell_pack(to(h), T, C)
    assert status == twell.TWELL_OK and 0 < hy.n_dense_host() < n
    nan = lambda *s, dt=torch.float32: torch.full(s, float("nan"), dtype=dt, device="cuda")
    out = twell.Grads(nan(n, dm, dt=dtype), nan(dff, dm), nan(dff), nan(dff, dm))
    g = twell.ffn_sparse_backward_act8(x8, to(wu), to(wd), hy, to(dy), out=out)
    torch.cuda.synchronize()
    x = act8_decode(x8.codes.cpu().numpy(), x8.scales.cpu().numpy(), dm)
    ref = oracle.ffn_backward_from_h(x, h.astype(np.float64), *(a.astype(np.float64)
                                                               for a in (wu, wd, dy)))
    assert max(np.abs(a).max() for a in (ref.dw_down, ref.dw_up_t, ref.db, ref.dx)) < 2 ** 24
    np.testing.assert_array_equal(as_f64(g.dw_down), ref.dw_down)
    np.testing.assert_array_equal(as_f64(g.dw_up_t), ref.dw_up_t)
    np.testing.assert_array_equal(as_f64(g.db_up), ref.db)
    np.testing.assert_array_equal(as_f32(g.dx), as_f32(torch.from_numpy(ref.dx).to(dtype)))
