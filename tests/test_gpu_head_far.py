"""The output head's float32 products of many rows far from the unit range: the powers of two by
which x and w are scaled are undone without leaving float32's range on the way.

z's bound is test_gpu_head's, and d 2^-133 beside it: where the scales together would pass 2^126,
x's is held back, so that x's parts are within 2^-25 of scaled values that meet w's of up to
2^15, and w's within 2^-25 of x's (each product off by 2^-9 at most); what undoes the scales is
then below 2^-125, and the sum's own cuts are within the relative part of the bound."""
import numpy as np
import pytest
import torch

from gpu_helpers import as_f64, say
from oracle.train_oracle import head_logprob
from test_gpu_head import backward, errors_of_z, forward, make, within

pytestmark = pytest.mark.gpu
# n, vocab, d: tiles past the vocabulary's end, whole tiles alone, many tiles
SIZES = [(70, 300, 64), (130, 1000, 72), (65, 256, 64), (1000, 9000, 72)]


def far(n, v, d, x_by, w_by, scale):
    m = make(n + v, n, v, d, torch.float32, scale)
    m["x"] *= 2.0 ** x_by
    m["w"] *= 2.0 ** w_by
    return m


def check_forward(m):
    x, w, t = as_f64(m["x"]), as_f64(m["w"]), m["t"].numpy()
    scale = float(np.float32(m["scale"]))
    logp, lse, stats, _ = head_logprob(x, w, t, scale)
    e_row = errors_of_z(x, w, scale).max(axis=1) + x.shape[1] * 2.0 ** -133
    got = forward(m)
    torch.cuda.synchronize()
    tol = 2 * e_row + 2.0 ** -20 * (1 + np.abs(lse))
    within("lse", got.lse, lse, tol)
    within("logp", got.logp, logp, tol)
    within("max", got.stats[:, 0], stats[:, 0], e_row)
    within("sum", got.stats[:, 1], stats[:, 1], stats[:, 1] * (2 * tol))
    return got


@pytest.mark.parametrize("n,v,d", SIZES)
@pytest.mark.parametrize("x_by,w_by,scale", [
    (-66, -66, 1.0),            # every z under 2^-126
    (-90, 0, 2.0 ** -40),       # rows of x far below
    (0, -90, 2.0 ** -40),
    (-40, -60, 0.7),            # what undoes the scales near float32's smallest
    (-70, 118, 0.8 * 2.0 ** -49),  # z of ordinary size behind scale * x out of range below
    (-100, 118, 0.8 * 2.0 ** -20),
    (44, -80, 2.0 ** 100),      # and above, z about 2^64 (dlogp keeps dw in range)
    (50, 60, 2.0 ** -110),
])
def test_scaled_operands(n, v, d, x_by, w_by, scale):
    say(f"head far n={n} v={v} d={d} x 2^{x_by} w 2^{w_by} scale {scale:.2e}")
    m = far(n, v, d, x_by, w_by, scale)
    if scale > 1:
        m["dlogp"] /= scale
    grads = backward(m, check_forward(m).stats)
    assert torch.isfinite(grads.dx).all() and torch.isfinite(grads.dw).all()


@pytest.mark.parametrize("n,v,d", SIZES)
def test_rows_of_far_sizes_side_by_side(n, v, d):
    """Rows of x of sizes from 2^-126 on beside w of 2^-60: each keeps its own scale."""
    say(f"head rows of far sizes n={n} v={v} d={d}")
    m = far(n, v, d, 0, -60, 1.0)
    m["x"] = (m["x"].double() * 2.0 ** torch.linspace(-126, 58, n).round().double()[:, None]).float()
    check_forward(m)
