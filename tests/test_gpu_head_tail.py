"""The output head's gradient at tokens that are unlikely in every row.

float32, more than 64 rows: dl / (scale dlogp) enters the products as two half-precision parts of it
times 2^15, whose steps end at 2^-24: it is within 2^-25 / 2^15 = 2^-40, and 2^-23 of itself.
float32, up to 64 rows: 24 bits of whatever size.  bfloat16: 8 bits of whatever size (half a step is
2^-8 of the value), 16 with up to 16 rows and vocab * d_model up to 2^25.  One row has a target and z = -k log 2 for k from 0 to 60, so that a row of dw is one dl
times x."""
import numpy as np
import pytest
import torch

from gpu_helpers import as_f64, say
from oracle.train_oracle import head_logprob
from test_gpu_head import U, backward, forward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,v,dtype,least,part", [
    (70, 700, torch.float32, 2.0 ** -40, 2.0 ** -22), (600, 700, torch.float32, 2.0 ** -40, 2.0 ** -22),
    (64, 700, torch.float32, 0.0, 2.0 ** -22), (5, 700, torch.float32, 0.0, 2.0 ** -22),
    (70, 700, torch.bfloat16, 0.0, 2.0 ** -8), (17, 700, torch.bfloat16, 0.0, 2.0 ** -8),
    (16, 700, torch.bfloat16, 0.0, 2.0 ** -16), (1, 700, torch.bfloat16, 0.0, 2.0 ** -16),
    (16, 1 << 19, torch.bfloat16, 0.0, 2.0 ** -16), (3, 1 << 19, torch.bfloat16, 0.0, 2.0 ** -16),
    (16, (1 << 19) + 1, torch.bfloat16, 0.0, 2.0 ** -8)])
def test_unlikely_tokens(n, v, dtype, least, part):
    say(f"head unlikely tokens n={n} v={v} {dtype}")
    d = 64
    gen = torch.Generator().manual_seed(n)
    live = n // 2
    x = torch.randn((n, d), generator=gen).to(dtype)
    x[live] = (1 + torch.rand(d, generator=gen)).to(dtype)
    x[live, 0] = 1
    w = torch.zeros((v, d), dtype=dtype)
    w[:, 0] = (-np.log(2.0) * (torch.arange(v) % 61).double()).to(dtype)
    t = torch.full((n,), -1)
    t[live] = 3
    m = dict(x=x, w=w, t=t, scale=1.0, dlogp=torch.full((n,), 0.75))
    got = as_f64(backward(m, forward(m).stats).dw[:700])
    z = (as_f64(x[live])[None] @ as_f64(w).T)
    p = np.exp(z - head_logprob(as_f64(x[live])[None], as_f64(w), np.array([3]), 1.0)[1])[0]
    dl = -p[:700]
    dl[3] += 1
    # z is exact but for float32's roundings of its parts' products, 2^-21 of it; the exponential's,
    # the sum's and the maximum's beside
    e_p = p[:700] * (2.0 ** -21 * np.abs(z[0]).max() + 2.0 ** -20)
    xs = as_f64(x[live])
    tol = 0.75 * (e_p + np.maximum(np.abs(dl) * part * (1 + 2.0 ** -6), least))[:, None] * xs
    ref = 0.75 * dl[:, None] * xs
    step = torch.finfo(dtype).eps / 2
    # x's own parts and the result's rounding
    off = np.abs(got - ref) - tol - np.abs(ref) * (2.0 ** -22 + step * 1.01) - least * 2.0 ** -22
    assert np.all(off <= 0), float((off / (0.75 * xs)).max())
