"""The norms with several rows to a workgroup, one after another in the same LDS: the forward pass
takes two from 4096 workgroups' steps on (four rows each up to 1024 columns), the gradient deals its
rows to 512 workgroups (256 past 4096 columns).  Every choice of what is given, since the barriers
between two rows depend on it.  Bounds: test_gpu_norm's."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_norm import ALL, BOTH, FORMS, check_backward, check_forward, make, run_forward

pytestmark = pytest.mark.gpu
EVERY = [ALL, *FORMS]
SOME = [ALL, dict(ALL, post=False), dict(ALL, pre=False), dict(ALL, post=False, pre=False)]
FORWARD = ([(4099, 1032, f) for f in EVERY] + [(4097, 2056, f) for f in SOME]
           + [(4097, 4104, f) for f in SOME] + [(4098, 8200, ALL), (4097, 8200, SOME[1])]
           + [(16389, 16, f) for f in SOME] + [(16387, 520, f) for f in SOME])
BACKWARD = ([(1101, 1032, f) for f in EVERY] + [(1029, 2056, f) for f in EVERY]
            + [(600, 4104, f) for f in SOME] + [(520, 8200, f) for f in SOME]
            + [(4111, 264, f) for f in SOME])


def alpha_of(form):
    return 0.8 if form["y"] else 1.0


@BOTH
@pytest.mark.parametrize("n,d,form", FORWARD)
def test_forward(n, d, form, dtype):
    say(f"norm forward rows {dtype} {n}x{d} {form}")
    m = make(n + d, n, d, dtype, **form)
    got = run_forward(m, alpha_of(form))
    torch.cuda.synchronize()
    check_forward(got, m, alpha_of(form))


@BOTH
@pytest.mark.parametrize("n,d,form", BACKWARD)
def test_backward(n, d, form, dtype):
    say(f"norm backward rows {dtype} {n}x{d} {form}")
    check_backward(make(n + d, n, d, dtype, **form), alpha_of(form))


@BOTH
def test_repeats(dtype):
    """The same bits again: no row reads what the one before left in LDS."""
    from activation_sparse_transformer_amd import twell
    for form in SOME:
        m = {k: v if v is None else v.cuda() for k, v in make(5, 4099, 4104, dtype, **form).items()}
        w = {k: m[k] for k in ("w_post", "gate", "w_pre")}
        f = lambda: twell.twell_norm_forward(m["residual"], m["y"], **w)
        b = lambda: twell.twell_norm_backward(m["residual"], m["y"], m["dr"], m["dx"], **w)
        for call in (f, b):
            first = vars(call())
            for _ in range(3):
                again = vars(call())
                assert all(v is None or torch.equal(v, again[k]) for k, v in first.items())
