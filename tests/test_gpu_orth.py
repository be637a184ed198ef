"""GPU parity of twell_orthogonalize against the CPU oracle, which iterates the polynomial on the
singular values in float64.

Compared by 2-norms of whole matrices.  One step's own error: X, G and B are held as two
half-precision parts (2^-23), their products leave out 2^-22 at most, and the float32 sums behind
them add under 50 roundings of 2^-24 (independent ones, as their root), so a step is within
r = 2^-18 of its result.  An error of X grows by at most max |f'| of f(s) = a s + b s^3 + c s^5 over
the singular values, 3.9 on [0, 1.2] for the usual coefficients: after k steps r (3.9^k - 1) / 2.9,
times 1.2 as f overshoots 1.
A bfloat16 matrix's X is rounded to 11 bits besides, by at most 2^-11 (0.29 of an ulp, 2^-11 to
2^-10, in the mean) of each element in every step, and the output to 8.  That grows like any other
change of X; growth of a real change is found by the oracle itself: a matrix whose elements are
changed at random by up to 2^-8 (M's own rounding) moves by c, and an X changed in every step by an
eighth of that moves by less than sqrt(k) / 8 of the largest move of k and fewer steps.  Twice that
is allowed, for the luck of the one change tried."""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import as_f64, say
from oracle.train_oracle import orthogonalize

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
COEFF = (3.4445, -4.775, 2.0315)
AS_F32 = tuple(float(np.float32(c)) for c in COEFF)


def make(seed, rows, cols, dtype, size=1e-3):
    g = torch.Generator().manual_seed(seed)
    k = min(4, rows, cols)
    m = torch.randn((rows, cols), generator=g)
    m += 2 * torch.randn((rows, k), generator=g) @ torch.randn((k, cols), generator=g)
    return (m * size).to(dtype)


def bound(m, steps, coefficients=AS_F32):
    """The relative error allowed of m's result."""
    r = 2.0 ** -18
    grown = r if steps == 1 else 1.2 * r * (3.9 ** steps - 1) / 2.9
    if m.dtype == torch.float32:
        return grown
    x = as_f64(m)
    change = 1 + 2.0 ** -8 * np.random.default_rng(0).uniform(-1, 1, x.shape)
    moves = []
    for k in range(1, steps + 1):
        a, b = (orthogonalize(y, k, coefficients, 1e-7, 1.0) for y in (x, x * change))
        moves.append(np.linalg.norm(b - a) / np.linalg.norm(a))
    return grown + 2 * np.sqrt(steps) / 8 * max(moves) + torch.finfo(m.dtype).eps / 2


def check(m, steps=5, scale=1.0, got=None):
    if got is None:
        got = twell.twell_orthogonalize(m.cuda(), steps=steps, scale=scale)
    ref = orthogonalize(as_f64(m), steps, AS_F32, float(np.float32(1e-7)), float(np.float32(scale)))
    off = np.linalg.norm(as_f64(got) - ref) / np.linalg.norm(ref)
    tol = bound(m, steps)
    say(f"off {off:.2e} of {tol:.2e}")
    assert off <= tol
    return got


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [
    (1, 1), (1, 7), (5, 1), (3, 3), (16, 40), (64, 64), (65, 63), (33, 500), (100, 257), (500, 33),
    (128, 512), (127, 1024), (129, 300), (1030, 128), (128, 8192), (8200, 60), (64, 40000),
    (513, 130), (256, 1000), (700, 300), (1025, 511), (40, 5000), (2100, 70)])
def test_matches_oracle(rows, cols, dtype):
    say(f"orthogonalize {dtype} {rows}x{cols}")
    m = make(rows + cols, rows, cols, dtype)
    check(m, 1)
    check(m, 5, 0.2)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [(1300, 4200), (4100, 1100)])
def test_larger(rows, cols, dtype):
    check(make(7, rows, cols, dtype), 1)
    check(make(8, rows, cols, dtype), 3)


@pytest.mark.gpu
@BOTH
def test_other_coefficients(dtype):
    """The cubic iteration 1.5 s - 0.5 s^3, whose steps do not overshoot."""
    m = make(3, 70, 200, dtype)
    c = (1.5, -0.5, 0.0)
    got = twell.twell_orthogonalize(m.cuda(), steps=7, coefficients=c)
    ref = orthogonalize(as_f64(m), 7, c, float(np.float32(1e-7)), 1.0)
    off = np.linalg.norm(as_f64(got) - ref) / np.linalg.norm(ref)
    assert off <= 2.0 ** -18 * (1.5 ** 7 - 1) / 0.5 if dtype == torch.float32 else bound(m, 7, c)


@pytest.mark.gpu
@BOTH
def test_far_sizes(dtype):
    """The norm is summed in double: no square leaves its range."""
    m = make(5, 40, 90, dtype, 1.0)
    ref = twell.twell_orthogonalize(m.cuda())
    for e in (100, -30):  # beside these sizes eps is nothing
        big = m * 2.0 ** e
        got = twell.twell_orthogonalize(big.cuda(), eps=1e-30)
        assert (got - ref).double().norm() <= 2 * bound(m, 5) * ref.double().norm()


@pytest.mark.gpu
@BOTH
def test_zero_nan_and_infinity(dtype):
    z = torch.zeros((70, 40), dtype=dtype, device="cuda")
    assert not twell.twell_orthogonalize(z).any()
    for bad in (float("nan"), float("inf")):
        z[3, 3] = bad
        assert torch.isnan(twell.twell_orthogonalize(z)).all()


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [(90, 200), (300, 130)])
def test_in_place_replayed_and_on_another_stream(rows, cols, dtype):
    m = make(9, rows, cols, dtype).cuda()
    ref = twell.twell_orthogonalize(m)
    here = m.clone()
    assert twell.twell_orthogonalize(here, out=here) is here and torch.equal(here, ref)
    ws = twell.orthogonalize_workspace(rows, cols, dtype, "cuda")
    out = torch.empty_like(m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        twell.twell_orthogonalize(m, out=out, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        twell.twell_orthogonalize(m, out=out, workspace=ws)
    for _ in range(3):
        out.fill_(3)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


# ------------------------------------------------------------------ host only
def test_oracle_hand_worked():
    """A diagonal matrix's singular values, one step by hand; any matrix by its products."""
    got = orthogonalize(np.diag([3.0, 4.0]), 1, (2.0, -1.5, 0.5), 0.0, 2.0)
    f = lambda s: 2 * s - 1.5 * s ** 3 + 0.5 * s ** 5
    np.testing.assert_allclose(got, 2 * np.diag([f(0.6), f(0.8)]), atol=1e-14)
    for rows, cols in ((5, 9), (9, 5)):
        m = np.random.default_rng(1).normal(size=(rows, cols))
        x = m / (np.linalg.norm(m) + 0.1)
        for _ in range(3):
            g = x @ x.T
            x = COEFF[0] * x + (COEFF[1] * g + COEFF[2] * g @ g) @ x
        np.testing.assert_allclose(orthogonalize(m, 3, COEFF, 0.1, 1.0), x, atol=1e-12)


P = 4096  # an aligned address that no call below reads
BAD, UNSUPPORTED = twell.TWELL_ERR_INVALID_ARG, twell.TWELL_ERR_UNSUPPORTED


def shape(**kw):
    s = dict(rows=64, cols=128, dtype=0, steps=5, a=3.0, b=-4.0, c=2.0, eps=1e-7, scale=1.0)
    return ctypes.byref(twell.OrthShape(*{**s, **kw}.values()))


def test_refused_shapes():
    lib = twell.load()
    nan, inf = float("nan"), float("inf")
    for kw in (dict(rows=0), dict(cols=-1), dict(dtype=2), dict(steps=0), dict(steps=65),
               dict(a=nan), dict(b=inf), dict(c=-inf), dict(scale=nan), dict(eps=0.0),
               dict(eps=-1.0), dict(eps=inf), dict(eps=nan)):
        assert lib.twell_orthogonalize(shape(**kw), None, None, None, 0, None) == BAD, kw
        assert lib.twell_orthogonalize_workspace_size(shape(**kw)) == 0
    for kw in (dict(rows=(1 << 20) + 1), dict(cols=(1 << 20) + 1), dict(rows=65537, cols=65537),
               dict(rows=65536, cols=65537)):
        assert lib.twell_orthogonalize(shape(**kw), None, None, None, 0, None) == UNSUPPORTED, kw
    assert lib.twell_orthogonalize(None, P, P, P, 1 << 40, None) == BAD
    # the largest matrices are counted without overflow
    assert lib.twell_orthogonalize_workspace_size(shape(rows=65536, cols=65536)) > 1 << 34
    assert lib.twell_orthogonalize_workspace_size(shape(rows=1 << 20, cols=1 << 12)) > 1 << 34


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="fake device pointers are passed only on a GPU-less host")
def test_refused_pointers():
    lib = twell.load()
    for p in ((None, P, P), (P, None, P), (P, P, None), (P + 8, P, P), (P, P + 8, P), (P, P, P + 8)):
        assert lib.twell_orthogonalize(shape(), *p, 1 << 40, None) == BAD
    assert lib.twell_orthogonalize(shape(), P, P, P, 64, None) == twell.TWELL_ERR_WORKSPACE


def test_refused_tensors():
    m = torch.zeros((8, 8))
    f = twell.twell_orthogonalize
    for bad in (lambda: f(m), lambda: f(m.half()), lambda: f(m.double()), lambda: f(m[:, :4]),
                lambda: f(m, out=torch.zeros((8, 9))), lambda: f(m, out=m.bfloat16())):
        with pytest.raises(ValueError):
            bad()
    big = torch.empty((1, 2 ** 32 + 1), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        f(big)
    with pytest.raises(twell.TwellError):
        twell.orthogonalize_workspace(1 << 21, 4, torch.float32, "meta")
