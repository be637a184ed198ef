"""twell_orthogonalize on the kernels that large matrices take (256 x 256 tiles, whose update ends in
the product's epilogue), with coefficients, sizes and values away from the usual ones on both sides
of the shorter side's 128.

Bounds as in test_gpu_orth: a float32 step is within r = 2^-18 of its result, and an error of X grows
by at most max |f'| over the singular values; a bfloat16 X of 11 bits in each of k steps moves by
less than sqrt(k) / 8 of what M's own rounding moves it by, twice that is allowed, and the output's
half step beside it."""
import numpy as np
import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import as_f64, say
from oracle.train_oracle import orthogonalize
from test_gpu_orth import AS_F32, BOTH, COEFF, bound, make

# every product of these takes 256 x 256 tiles in both types (test_cut_rules.py)
BIG = [(2183, 5283), (5283, 2183), (2829, 2821)]
# shorter sides on both sides of 128, 128 x 128 tiles
SHORT, LONG = (70, 200), (200, 700)


def by_products(m, steps, coefficients, eps):
    """The steps in float64 on the GPU (the oracle's hand-worked test holds the same products)."""
    a, b, c = coefficients
    x = m.double().cuda()
    x = (x.t() if x.shape[0] > x.shape[1] else x).contiguous()
    x = x / (x.square().sum().sqrt() + eps)
    for _ in range(steps):
        g = torch.matmul(x, x.t().contiguous())
        x = a * x + torch.matmul(b * g + c * torch.matmul(g, g), x)
    return x.t() if m.shape[0] > m.shape[1] else x


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", BIG)
@pytest.mark.parametrize("steps", [1, 2, 3])
def test_large_tiles(rows, cols, steps, dtype):
    say(f"orthogonalize {dtype} {rows}x{cols} steps {steps}")
    m = make(rows + steps, rows, cols, dtype)
    got = twell.twell_orthogonalize(m.cuda(), steps=steps).double()
    f = lambda x, k: by_products(x, k, AS_F32, float(np.float32(1e-7)))
    ref = f(m, steps)
    off = float((got - ref).norm() / ref.norm())
    r = 2.0 ** -18
    tol = r if steps == 1 else 1.2 * r * (3.9 ** steps - 1) / 2.9
    if dtype == torch.bfloat16:
        g = torch.Generator().manual_seed(0)
        other = m.double() * (1 + 2.0 ** -8 * (2 * torch.rand(m.shape, generator=g).double() - 1))
        moves = []
        for k in range(1, steps + 1):
            a, b = f(m, k), f(other, k)
            moves.append(float((a - b).norm() / a.norm()))
        tol += 2 * np.sqrt(steps) / 8 * max(moves) + torch.finfo(dtype).eps / 2
    say(f"off {off:.2e} of {tol:.2e}")
    assert off <= tol


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [(130, 300), (500, 1300), (700, 300), (1300, 1100)])
def test_two_steps(rows, cols, dtype):
    """The update's first step leaves X in two parts: with one lost, 2^-12 of it would be off."""
    m = make(rows, rows, cols, dtype)
    got = twell.twell_orthogonalize(m.cuda(), steps=2).double()
    ref = by_products(m, 2, AS_F32, float(np.float32(1e-7)))
    off = float((got - ref).norm() / ref.norm())
    assert off <= bound(m, 2)  # 2^-15.5 in float32


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [SHORT, LONG, (700, 200), (300, 130)])
def test_cubic(rows, cols, dtype):
    """1.5 s - 0.5 s^3, whose steps do not overshoot and whose |f'| is at most 1.5."""
    m = make(3, rows, cols, dtype)
    c = (1.5, -0.5, 0.0)
    got = twell.twell_orthogonalize(m.cuda(), steps=7, coefficients=c)
    eps = float(np.float32(1e-7))
    x = as_f64(m)
    ref = orthogonalize(x, 7, c, eps, 1.0)
    off = np.linalg.norm(as_f64(got) - ref) / np.linalg.norm(ref)
    tol = 2.0 ** -18 * (1.5 ** 7 - 1) / 0.5
    if dtype == torch.bfloat16:
        change = 1 + 2.0 ** -8 * np.random.default_rng(0).uniform(-1, 1, x.shape)
        moves = []
        for k in range(1, 8):
            a, b = (orthogonalize(y, k, c, eps, 1.0) for y in (x, x * change))
            moves.append(np.linalg.norm(b - a) / np.linalg.norm(a))
        tol += 2 * np.sqrt(7) / 8 * max(moves) + torch.finfo(dtype).eps / 2
    say(f"off {off:.2e} of {tol:.2e}")
    assert off <= tol


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [SHORT, LONG])
def test_growing_coefficients(rows, cols, dtype):
    """Two steps that take X to 1e20 and G to 1e8: the scales follow.  The last step is 1e4 s - s^3 +
    s^5 at s up to 1e4: an error of X grows fivefold, the step's own is r."""
    m = make(4, rows, cols, dtype)
    c = (1e4, -1.0, 1.0)
    got = twell.twell_orthogonalize(m.cuda(), steps=2, coefficients=c)
    ref = orthogonalize(as_f64(m), 2, c, float(np.float32(1e-7)), 1.0)
    off = np.linalg.norm(as_f64(got) - ref) / np.linalg.norm(ref)
    x = 0 if dtype == torch.float32 else 6 * 2.0 ** -11 + 2.0 ** -8  # X's 11 bits, the output's 8
    assert off <= 6 * 2.0 ** -18 + x


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [SHORT, LONG])
@pytest.mark.parametrize("coefficients,steps", [((2.0 ** 30, 0.0, 0.0), 4), ((1e30, 1e30, 1e30), 3),
                                                ((3e38, -3e38, 3e38), 64), ((0.0, 0.0, 3e38), 2)])
def test_coefficients_out_of_range(rows, cols, coefficients, steps, dtype):
    """X, G or B past 2^100: infinities and NaN, or the right value, never another number."""
    m = make(5, rows, cols, dtype)
    c = tuple(float(np.float32(v)) for v in coefficients)
    got = as_f64(twell.twell_orthogonalize(m.cuda(), steps=steps, coefficients=c))
    with np.errstate(over="ignore", invalid="ignore"):
        ref = orthogonalize(as_f64(m), steps, c, float(np.float32(1e-7)), 1.0)
    fine = np.isfinite(got)
    if fine.any():
        assert np.isfinite(ref).all()
        off = np.linalg.norm((got - ref)[fine]) / np.linalg.norm(ref)
        assert off <= 2.0 ** -7


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("coefficients", [(0.1, 0.0, 0.0), (0.0, 0.0, 0.0), (0.0, 0.5, 0.0),
                                          (1.0, 0.0, 0.0)])
@pytest.mark.parametrize("rows,cols", [SHORT, LONG])
def test_shrinking_coefficients(rows, cols, coefficients, dtype):
    """X down to 1e-4 and its cube.  X's parts carry an error of 2^-38 of the bound of X's singular
    values, which for the cube is far above them: it is allowed for every element."""
    m = make(6, rows, cols, dtype)
    c = tuple(float(np.float32(v)) for v in coefficients)
    got = as_f64(twell.twell_orthogonalize(m.cuda(), steps=4, coefficients=c))
    ref = orthogonalize(as_f64(m), 4, c, float(np.float32(1e-7)), 1.0)
    # s^3 triples an error at every step: (3^4 - 1) / 2 = 40 r; a bfloat16 X is off by 2^-11 in
    # every step, 40 of them
    tol = 40 * (2.0 ** -18 if dtype == torch.float32 else 2.0 ** -11) + (
        0 if dtype == torch.float32 else 2.0 ** -8)
    most = 1.0  # of |a s + b s^3| over [0, 1], step by step: these grow with s
    for _ in range(4):
        most = c[0] * most + c[1] * most ** 3
    least = np.sqrt(got.size) * 2.0 ** -38 * most
    assert np.linalg.norm(got - ref) <= tol * np.linalg.norm(ref) + least


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [SHORT, LONG, (300, 130)])
def test_far_sizes(rows, cols, dtype):
    m = make(7, rows, cols, dtype, 1.0)
    ref = twell.twell_orthogonalize(m.cuda())
    for e in (100, -30):  # beside these sizes eps is nothing
        got = twell.twell_orthogonalize((m * 2.0 ** e).cuda(), eps=1e-30)
        assert (got - ref).double().norm() <= 2 * bound(m, 5) * ref.double().norm()


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", [SHORT, LONG, (300, 130), (1100, 2100)])
@pytest.mark.parametrize("steps", [1, 2])
def test_zero_nan_and_infinity(rows, cols, steps, dtype):
    z = torch.zeros((rows, cols), dtype=dtype, device="cuda")
    assert not twell.twell_orthogonalize(z, steps=steps).any()
    m = make(8, rows, cols, dtype).cuda()
    for bad in (float("nan"), float("inf"), -float("inf")):
        m[rows - 1, cols // 2] = bad
        assert torch.isnan(twell.twell_orthogonalize(m, steps=steps)).all()


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("rows,cols", BIG[:1] + [(978, 2283)])
def test_repeats(rows, cols, dtype):
    """The same bits again, whatever the workspace held."""
    m = make(9, rows, cols, dtype).cuda()
    ws = twell.orthogonalize_workspace(rows, cols, dtype, "cuda")
    first = twell.twell_orthogonalize(m, workspace=ws).clone()
    for fill in (0, 255, 63):
        ws.fill_(fill)
        assert torch.equal(twell.twell_orthogonalize(m, workspace=ws), first)
