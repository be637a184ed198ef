"""Logits far past 2^24, where z itself is known to no unit: the largest of a row has the
probability 1 and nothing is infinite or NaN, whatever the scale's bits."""
import numpy as np
import pytest
import torch

from gpu_helpers import as_f64, say
from oracle.train_oracle import head_logprob
from test_gpu_head import U, backward, errors_of_z, forward, make, root_sum, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,v,d", [(5, 300, 64), (24, 1000, 64), (70, 300, 64), (300, 5000, 72)])
@pytest.mark.parametrize("by", [24, 30, 34, 64, 100])
def test_logits_past_the_unit(n, v, d, by, dtype):
    """Compared where a row's largest z stands out by more than the error of both, so that p is 1
    there and 0 elsewhere, exactly; dx where the gradient sums z as the forward pass did (24 rows in
    bfloat16 are few rows to the one, many to the other)."""
    say(f"head logits about 2^{by} {dtype} n={n} v={v} d={d}")
    m = make(by + n, n, v, d, dtype, 0.7 * 2.0 ** by)
    x, w, t = as_f64(m["x"]), as_f64(m["w"]), m["t"].numpy()
    scale = float(np.float32(m["scale"]))
    logp, lse, stats, z = head_logprob(x, w, t, scale)
    ez = errors_of_z(x, w, scale).max(axis=1)
    top2 = np.sort(z, axis=1)[:, -2:]
    clear = top2[:, 1] - top2[:, 0] > 2 * ez + 100
    assert clear.mean() > 0.6
    got = forward(m)
    grads = backward(m, got.stats)
    torch.cuda.synchronize()
    within("max", got.stats[:, 0], stats[:, 0], ez)
    within("lse", got.lse, lse, ez + 2.0 ** -20 * (1 + np.abs(lse)))
    within("logp", got.logp, logp, 2 * ez + 2.0 ** -20 * (1 + np.abs(lse)))
    s = as_f64(got.stats[:, 1])
    assert np.all(s[clear] == 1) and np.all((s >= 1) & (s <= v))
    ok = (t >= 0) & (t < v)
    g = np.where(ok, as_f64(m["dlogp"]) * scale, 0.0)
    dl = np.where(z == z.max(axis=1)[:, None], -g[:, None], 0.0)
    dl[np.arange(n)[ok], t[ok]] += g[ok]
    # a dl is g, -g or 0: with bfloat16 operands rounded by half a step
    step = torch.finfo(dtype).eps / 2
    part = step if dtype == torch.bfloat16 else 2 * U
    sums = 24 * np.sqrt(1.5 * v) * U
    tol = (part * np.abs(dl)) @ np.abs(w) + sums * root_sum(dl, w.T)
    dx = dl @ w
    off = np.abs(as_f64(grads.dx) - dx) - tol - step * np.abs(dx) * 1.01
    if n != 24 or dtype == torch.float32:
        assert np.all(off[clear | ~ok] <= 0)
    assert np.all(np.abs(as_f64(grads.dx)) <= 2 * np.abs(g)[:, None] * np.abs(w).max() * (1 + 4 * step))
    # every p is within [0, 1] (and a row's sum within its rounding), so dw stays under these
    most = np.abs(g) @ np.where(ok[:, None], np.abs(x), 0.0)
    assert np.all(np.abs(as_f64(grads.dw)) <= most * (1 + 4 * step))
