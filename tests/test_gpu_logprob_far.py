"""The log-probability gradient where float32 log-sum-exps are coarse or out of range: rows past
|lse| = 128 that span several workgroups' chunks, in place and not, and rows of the type's lowest
value under a scale above 1, whose scaled logits leave float32.

Tolerances are those of the ordinary rows (test_gpu_logprob.py): a gradient element within 1e-5 of
(|dlogp| + |dentropy| (1 + entropy)) * scale, plus its rounding to bfloat16."""
import numpy as np
import pytest
import torch

from gpu_helpers import as_f64, say
from test_gpu_logprob import check_backward, odd_rows, run_backward

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("v", [20011, 70000])
@pytest.mark.parametrize("ent", [True, False])
@pytest.mark.parametrize("form", ["same rows", "shifted rows", "in place"])
def test_far_rows_of_several_chunks(form, ent, v, dtype):
    """A row's chunks (8192 bfloat16 or 4096 float32 columns) belong to different workgroups."""
    say(f"logprob grad far rows {dtype} v={v} ent={ent} {form}")
    x, t = odd_rows(v, dtype)
    t[4] = 1
    keep = [r for r in range(16) if r not in (13, 14)]
    dlogp = torch.linspace(-1, 2, 16)
    dent = torch.linspace(1, -1, 16) if ent else None
    f, got = run_backward(x, t, 1.0, dlogp, dent, v + 5, v + (6 if form == "shifted rows" else 5),
                          form == "in place")
    lse = as_f64(f.lse)
    assert (np.abs(lse[[1, 8, 11, 15]]) > 128).all()
    assert not got[0].any() and np.isnan(got[[13, 14]]).any(axis=1).all()
    check_backward(got[keep], x[keep], t[keep], 1.0, dlogp[keep], dent[keep] if ent else None,
                   as_f64(f.entropy)[keep])


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,v", [(6, 40), (6, 30000), (5000, 130)])
def test_lowest_values_under_a_scale_are_not_a_mask(n, v, dtype):
    """scale * lowest is below float32's range, yet such a row is uniform over its places; only
    rows of -inf have lse = -inf and no gradient."""
    say(f"logprob lowest values, scale 2: {dtype} n={n} v={v}")
    x = torch.full((n, v), torch.finfo(dtype).min, dtype=dtype)
    x[1::3] = -torch.inf            # nothing left
    x[2::3, ::2] = -torch.inf       # the odd places left
    t = torch.arange(n) % v
    t[2::3] = 1
    ones = torch.ones(n)
    f, got = run_backward(x, t, 2.0, ones, 0.5 * ones)
    lse, logp, entropy = (as_f64(a) for a in (f.lse, f.logp, f.entropy))
    left = np.array([v, 0, v // 2])[np.arange(n) % 3].astype(np.float64)
    live = left > 0
    np.testing.assert_array_equal(lse, np.where(live, np.finfo(np.float32).min, -np.inf))
    with np.errstate(divide="ignore"):
        want = np.log(left)
    np.testing.assert_allclose(logp[live], -want[live], rtol=2e-6)
    np.testing.assert_allclose(entropy[live], want[live], rtol=1e-5)
    assert (logp[~live] == -np.inf).all() and not entropy[~live].any()
    # uniform rows: the entropy's part is zero, so 2 (1[j = t] - 1 / left)
    ref = np.where(live[:, None] & (as_f64(x) != -np.inf), -1 / np.maximum(left, 1)[:, None], 0.0)
    ref[live, t.numpy()[live]] += 1
    tol = 2e-5 * (2 + np.where(live, want, 0))[:, None] + 2.0 ** -8 * np.abs(2 * ref) * (
        dtype == torch.bfloat16)
    assert np.all(np.abs(got - 2 * ref) <= tol), float(np.abs(got - 2 * ref).max())
    assert not got[~live].any()
