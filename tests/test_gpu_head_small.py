"""The gradient of the output head's float32 rows (more than 64) where w, x or scale * dlogp * x are
small: parts keep their bits down to float32's smallest normal numbers.

Bounds as test_gpu_head's for dx and dw.  The largest element of w and of scale * dlogp * x is
scaled to [2^14, 2^15) where 2^126 suffices, so that an element's parts are within 2^-25 of it
scaled: of a largest of 2^-126, which is scaled to 1, within 2^-25 of itself.  That error meets a
dl / (scale dlogp) of at most 1 per row.  What float32 cannot hold is beside it: half a step of
subnormal numbers, 2^-150, for each result and each scale * dlogp * x."""
import numpy as np
import pytest
import torch

from gpu_helpers import as_f64, say
from oracle.train_oracle import head_logprob, head_logprob_grad
from test_gpu_head import U, backward, errors_of_z, forward, make, root_sum, within

pytestmark = pytest.mark.gpu


def parts_error(largest):
    """Of an element in two half-precision parts, beside 2^-22.4 of itself."""
    e = min(14 - int(np.floor(np.log2(largest))), 126)
    return 2.0 ** (-25 - e)


def check(m):
    x, w, t = as_f64(m["x"]), as_f64(m["w"]), m["t"].numpy()
    scale = float(np.float32(m["scale"]))
    logp, lse, stats, z = head_logprob(x, w, t, scale)
    e_row = errors_of_z(x, w, scale).max(axis=1) + x.shape[1] * 2.0 ** -133
    got = backward(m, forward(m).stats)
    torch.cuda.synchronize()
    dlogp = as_f64(m["dlogp"])
    dx, dw, dl = head_logprob_grad(x, w, t, dlogp, scale)
    ok = (t >= 0) & (t < len(w))
    g = np.where(ok, np.abs(dlogp) * scale, 0.0)
    p = np.exp(z - lse[:, None])
    e_dl = g[:, None] * (p * (2 * e_row[:, None] + 2.0 ** -20) + 2.0 ** -39) + np.abs(dl) * 2 * U
    xm = np.where(ok[:, None], x, 0.0)
    sums = lambda k: 24 * np.sqrt(1.5 * k) * U
    tol_dx = (e_dl @ np.abs(w) + sums(len(w)) * root_sum(dl, w.T)
              + np.abs(dl).sum(axis=1)[:, None] * parts_error(np.abs(w).max()))
    within("dx", got.dx, dx, tol_dx + np.abs(dx) * U * 1.01 + 2.0 ** -150)
    unit = np.abs(dl) / np.where(g > 0, g, 1)[:, None]  # |dl| / g
    most = (np.abs(xm) * g[:, None]).max()
    tol_dw = (e_dl.T @ np.abs(xm) + sums(len(x)) * root_sum(dl.T, xm.T)
              + unit.sum(axis=0)[:, None] * (parts_error(most) + 2.0 ** -150))
    within("dw", got.dw, dw, tol_dw + np.abs(dw) * U * 1.01 + 2.0 ** -150)


@pytest.mark.parametrize("n,v,d", [(70, 300, 64), (130, 1000, 72), (1000, 900, 136)])
@pytest.mark.parametrize("w_by,x_by,g_by", [
    (-118, 0, 20), (-112, 20, 60), (-124, 60, 40),  # w far below 1
    (0, -60, -50), (0, -100, -15), (10, -110, 0),   # and scale * dlogp * x
    (-90, -30, 0), (-60, -60, 0)])
def test_small_operands(n, v, d, w_by, x_by, g_by):
    say(f"head small n={n} v={v} d={d} w 2^{w_by} x 2^{x_by} dlogp 2^{g_by}")
    m = make(n + v + d, n, v, d, torch.float32)
    m["x"] *= 2.0 ** x_by
    m["w"] *= 2.0 ** w_by
    m["dlogp"] *= 2.0 ** g_by
    check(m)


@pytest.mark.parametrize("n,v,d", [(70, 300, 64), (300, 700, 136)])
@pytest.mark.parametrize("g_by", [-20, -100, 0])
def test_weights_up_to_the_largest_number(n, v, d, g_by):
    """Weights of +-1.5 2^127: dl / g times them passes float32's range where dx does not."""
    say(f"head largest weights n={n} v={v} d={d} dlogp 2^{g_by}")
    m = make(n, n, v, d, torch.float32)
    sign = torch.full((v, 1), -1.0)
    m["t"] = torch.arange(n) % 50
    sign[:50] = 1
    m["w"] = sign * (1.25 + 0.25 * torch.rand((v, d), generator=torch.Generator().manual_seed(1)))
    m["w"] *= 2.0 ** 127
    m["x"] = (m["x"] / d ** 0.5).double().mul(2.0 ** -127).float()
    m["dlogp"] *= 2.0 ** g_by
    check(m)
