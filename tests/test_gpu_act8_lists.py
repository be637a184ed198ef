"""The lists that the backward from an 8-bit checkpoint makes of h, at the sizes where their
parts end: more stored dense rows than workgroups for them, rows of several chunks, bitmaps of
many words.  Layers of small integers, in which every float32 sum is exact (the largest is below
2^24), so results equal the oracle's bit for bit; dx is rounded once."""
import numpy as np
import pytest
import torch

import oracle
from activation_sparse_transformer_amd import twell
from gpu_helpers import as_f32, as_f64, say
from oracle.train_oracle import act8_decode


def ternary(rng, shape, zero):
    a = rng.integers(-1, 2, size=shape).astype(np.float32)
    a[rng.random(shape) < zero] = 0
    return a


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,dm,dff,T,C", [
    (5000, 128, 640, 64, 4),     # over 1024 dense rows, 79 words of 64 rows
    (70, 256, 16896, 128, 4),    # dense rows of several chunks, the last one partial
    (65, 128, 2112, 64, 8),      # one neuron slice of 64, one row in the last word
])
def test_lists_integer_valued_exact(n, dm, dff, T, C, dtype):
    say(f"backward_act8 lists {dtype} n={n} dff={dff}")
    rng = np.random.default_rng(n + dff)
    wu, wd, dy = (ternary(rng, s, 0.6) for s in ((dff, dm), (dff, dm), (n, dm)))
    # half of the rows too full for their tiles, a few empty, the others sparse
    share = np.where(rng.random(n) < 0.5, 0.15, 0.005)
    share[::13] = 0
    h = np.where(rng.random((n, dff)) < share[:, None], rng.integers(1, 4, size=(n, dff)), 0)
    h[min(1, n - 1), -1] = 3
    ht = torch.from_numpy(h.astype(np.float32)).to(dtype).cuda()
    x8 = twell.Act8.empty(n, dm, dtype, "cuda:0")
    x8.codes.zero_()
    x8.codes[:, :dm] = torch.from_numpy(ternary(rng, (n, dm), 0.5).astype(np.int8)).cuda()
    x8.scales.copy_(torch.from_numpy(
        rng.integers(1, 3, size=tuple(x8.scales.shape)).astype(np.float32)))
    hy, status = twell.twell_pack(ht, T, C)
    assert status == twell.TWELL_OK and hy.n_dense_host() > 0.4 * n
    to = lambda a: torch.from_numpy(a).to(dtype).cuda()
    g = twell.ffn_sparse_backward_act8(x8, to(wu), to(wd), hy, to(dy))
    torch.cuda.synchronize()
    x = act8_decode(x8.codes.cpu().numpy(), x8.scales.cpu().numpy(), dm)
    ref = oracle.ffn_backward_from_h(x, h.astype(np.float64), *(a.astype(np.float64)
                                                               for a in (wu, wd, dy)))
    assert max(np.abs(a).max() for a in (ref.dw_down, ref.dw_up_t, ref.db, ref.dx)) < 2 ** 24
    np.testing.assert_array_equal(as_f64(g.dw_down), ref.dw_down)
    np.testing.assert_array_equal(as_f64(g.dw_up_t), ref.dw_up_t)
    np.testing.assert_array_equal(as_f64(g.db_up), ref.db)
    np.testing.assert_array_equal(as_f32(g.dx), as_f32(torch.from_numpy(ref.dx).to(dtype)))
