"""The output head where columns of z are masked through w: by the type's lowest value and by
-infinity, for some tokens, whole tiles of them, and all but one."""
import numpy as np
import pytest
import torch

from gpu_helpers import as_f64, say
from oracle.train_oracle import head_logprob, head_logprob_grad
from test_gpu_head import U, backward, errors_of_z, forward, make, root_sum, within

pytestmark = pytest.mark.gpu


def masked(n, v, d, dtype, value, where):
    """x's first column is 1 and w's is 0, or `value` where masked; with no target there."""
    m = make(n + v, n, v, d, dtype)
    m["x"][:, 0] = 1
    m["w"][:, 0] = 0
    m["w"][where, 0] = value
    if value == -float("inf"):
        m["w"][where, 1:] = 0
    keep = np.setdiff1d(np.arange(v), np.arange(v)[where])
    t = m["t"].numpy()
    t[(t >= 0) & (t < v)] = keep[t[(t >= 0) & (t < v)] % len(keep)]
    return m, keep


WHERE = {"one": lambda v: [v // 2], "ends": lambda v: [0, v - 1], "tiles": lambda v: slice(100, 700),
         "most": lambda v: slice(1, v), "last": lambda v: slice(v - 1, v)}


def check(m, keep):
    """Against the tokens that are left: the masked ones have no weight and no gradient."""
    x, w, t = as_f64(m["x"]), as_f64(m["w"])[keep], m["t"].numpy()
    v = len(m["w"])
    ok = (t >= 0) & (t < v)
    place = np.full(v + 1, -1)
    place[keep] = np.arange(len(keep))
    tk = np.where(ok, place[np.clip(t, 0, v)], -1)
    logp, lse, stats, z = head_logprob(x, w, tk, 1.0)
    e_row = errors_of_z(x, w, 1.0).max(axis=1)
    tol = 2 * e_row + 2.0 ** -20 * (1 + np.abs(lse))
    got = forward(m)
    within("lse", got.lse, lse, tol)
    within("logp", got.logp, logp, tol)
    within("max", got.stats[:, 0], stats[:, 0], e_row)
    grads = backward(m, got.stats)
    dx, dw, dl = head_logprob_grad(x, w, tk, as_f64(m["dlogp"]), 1.0)
    gone = np.setdiff1d(np.arange(v), keep)
    assert not grads.dw[torch.from_numpy(gone)].any()
    step = torch.finfo(m["x"].dtype).eps / 2
    part = step if m["x"].dtype == torch.bfloat16 else 0.0
    g = np.where(ok, np.abs(as_f64(m["dlogp"])), 0.0)
    p = np.exp(z - lse[:, None])
    e_dl = g[:, None] * p * (2 * e_row[:, None] + 2.0 ** -20) + np.abs(dl) * (part + 2 * U)
    xm = np.where(ok[:, None], x, 0.0)
    sums = lambda k: 24 * np.sqrt(1.5 * k) * U
    within("dw", grads.dw[torch.from_numpy(keep)], dw, e_dl.T @ np.abs(xm) + sums(len(x)) * root_sum(dl.T, xm.T)
           + step * np.abs(dw) * 1.01 + 1e-37)
    if np.isfinite(as_f64(m["w"])).all():  # else 0 times infinity
        within("dx", grads.dx, dx, e_dl @ np.abs(w) + sums(len(w)) * root_sum(dl, w.T)
               + step * np.abs(dx) * 1.01 + 1e-37)


@pytest.mark.parametrize("where", list(WHERE))
@pytest.mark.parametrize("n,v,d", [(3, 1000, 64), (16, 1000, 64), (64, 5000, 72)])
def test_lowest_float32(n, v, d, where):
    """Up to 64 rows, where float32 operands keep their own exponents."""
    say(f"head masked by the lowest float32 n={n} v={v} {where}")
    m, keep = masked(n, v, d, torch.float32, torch.finfo(torch.float32).min, WHERE[where](v))
    check(m, keep)


@pytest.mark.parametrize("value", ["lowest", "-inf"])
@pytest.mark.parametrize("where", list(WHERE))
@pytest.mark.parametrize("n,v,d", [(3, 1000, 64), (16, 1000, 64), (33, 1000, 64), (300, 3000, 72),
                                   (1500, 9000, 136)])
def test_bfloat16(n, v, d, where, value):
    say(f"head masked bfloat16 n={n} v={v} {where} {value}")
    low = torch.finfo(torch.bfloat16).min if value == "lowest" else -float("inf")
    m, keep = masked(n, v, d, torch.bfloat16, low, WHERE[where](v))
    check(m, keep)


@pytest.mark.parametrize("n", [3, 64])
@pytest.mark.parametrize("value", [1.0, -1.0])
def test_largest_float32(n, value):
    """Finite elements up to float32's largest, in x and in w, with results in range (2^-108 is as
    small as an element may be for its three parts to hold 24 bits)."""
    m = make(n, n, 300, 64, torch.float32)
    big = torch.finfo(torch.float32).max * value
    m["x"][:, 5], m["w"][:, 5] = big, 0
    m["w"][::3, 5] = 2.0 ** -108
    m["x"][:, 6], m["w"][:, 6] = 2.0 ** -108, big
    x, w, t = as_f64(m["x"]), as_f64(m["w"]), m["t"].numpy()
    logp, lse, _, _ = head_logprob(x, w, t, 1.0)
    tol = 2 * errors_of_z(x, w, 1.0).max(axis=1) + 2.0 ** -20 * (1 + np.abs(lse))
    got = forward(m)
    within("lse", got.lse, lse, tol)
    within("logp", got.logp, logp, tol)
