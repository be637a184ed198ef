"""Which tiles the head's and the updates' products take (host only): the library's cost rules
written down a second time, held to the library by the workspace sizes that follow from them, and
the shapes of the GPU tests looked up in them, so that a change of the rules shows where a test no
longer reaches the kernels that it is for."""
import ctypes
import math

import pytest

from activation_sparse_transformer_amd import twell
from test_gpu_head_tiles import LARGE, MIXED
from test_gpu_orth_paths import BIG

SIDE = {"big": 256, "mid": 128}


def blocks(n, b):
    return -(-n // b)


def up64(v):
    return blocks(v, 64) * 64


def wide_cut(rows, cols, steps, most, triangle, whole):
    """(tile, slices, microseconds) of a product."""
    best = ("mid", 1, 1e300)
    for tile in ("big", "mid"):
        side = SIDE[tile]
        mb, nb = blocks(rows, side), blocks(cols, side)
        tiles = mb * (mb + 1) // 2 if triangle else mb * nb
        for s in range(1, min(most, max(steps // 4, 1)) + 1):
            each, groups = blocks(steps, s), tiles * s
            if tile == "big":
                us = blocks(groups, 256) * (each * 2.1 + 6)
            elif groups <= 256:
                us = each * 0.78 + 4
            else:
                us = blocks(groups, 512) * (each * 1.25 + 4)
            if s > 1 or not whole:
                us += s * tiles * side * side * 8 / 5e6
            if us < best[2]:
                best = (tile, s, us)
            if groups > 1024:
                break
    return best


def carved(*parts):
    return sum(blocks(p, 256) * 256 for p in parts)


# ------------------------------------------------------------------ updates (shorter side past 128)
def orth_cuts(rows, cols, eb):
    m, n = sorted((rows, cols))
    kinds = (3, 3) if eb == 4 else (1, 2)  # products of parts in X X^T and in B X
    return (wide_cut(m, m, up64(n) // 64 * kinds[0], 32, True, False),
            wide_cut(m, m, up64(m) // 64 * 3, 32, True, False),
            wide_cut(n, m, up64(m) // 64 * kinds[1], 32, False, True))


def orth_bytes(rows, cols, eb):
    m, n = sorted((rows, cols))
    square, whole = m * up64(m), m * up64(n)
    gram, sq, update = (c[1] for c in orth_cuts(rows, cols, eb))
    sums = max(max(gram, sq) * square, update * whole)
    return carved(512 * 8, 4 * whole, 4 * whole, 4 * square, 4 * square, 4 * sums)


# ------------------------------------------------------------------ the head of many rows
def equal_pieces(v, most):
    pieces = blocks(v, min(most, v))
    return min(blocks(blocks(v, pieces), 256) * 256, v)


def piece_of(v, per_column, budget, n, us):
    most = max(budget // per_column // 256 * 256, 1024)
    equal = equal_pieces(v, most)
    unit = 65536 // math.gcd(blocks(n, 256), 256)
    if equal >= v or most < unit:
        return equal
    filled = most // unit * unit
    total = lambda p: v // p * us(p) + (us(v % p) if v % p else 0)
    return filled if total(filled) < total(equal) else equal


def head_cuts(n, v, d, eb):
    """The cuts over a piece of the vocabulary, forward and gradient, with the pieces."""
    of = 3 if eb == 4 else 1
    part, ld = (2 if eb == 4 else 1), up64(d)
    stats = lambda c: wide_cut(c, n, blocks(d, 64) * of, 1, False, True)
    dw = lambda c: wide_cut(d, c, blocks(n, 64) * of, 1, False, True)
    dx = lambda c: wide_cut(d, n, up64(c) // 64 * of, 32, False, False)
    forward = v
    if eb == 4:
        forward = piece_of(v, 4 * ld, 128 << 20, n, lambda c: stats(c)[2])
    back = piece_of(v, 2 * part * n + (4 * ld if eb == 4 else 0), 192 << 20, n,
                    lambda c: stats(c)[2] + dw(c)[2] + dx(c)[2])
    return dict(forward=forward, back=back, stats=stats(forward), dl=stats(back), dw=dw(back),
                dx=dx(back))


def head_bytes(n, v, d, eb):
    c, ld = head_cuts(n, v, d, eb), up64(d)
    part = 2 if eb == 4 else 1
    tiles = blocks(v, SIDE[c["stats"][0]])
    forward = [8 * tiles * n, 4 * n]
    back = [2 * part * n * d, 2 * part * n * up64(c["back"]), 4 * c["dx"][1] * n * d]
    if eb == 4:
        forward += [8, 4 * n, 4 * ld * n, 4 * ld * c["forward"]]
        back += [8, 4 * n, 4 * ld * n, 4 * ld * c["back"]]
    return carved(*forward), carved(*back)


# ------------------------------------------------------------------ the tests
ORTH = [(129, 300), (200, 700), (1025, 511), (1300, 4200), (4100, 1100), (978, 2283), (8192, 2048),
        (14336, 4096), (4096, 14336), (20000, 700), (300, 100000), *BIG]
HEAD = [(65, 300, 1032), (70, 70000, 8), (200, 50000, 1024), (1000, 2900, 64), (4090, 5000, 40),
        (1100, 100000, 64), (2001, 49999, 1000), (4096, 32768, 2048), (257, 3, 2048), *LARGE, *MIXED]


@pytest.mark.parametrize("eb", [2, 4])
def test_the_rules_are_the_librarys(eb):
    lib = twell.load()
    dtype = 1 if eb == 2 else 0  # bfloat16, float32
    for rows, cols in ORTH:
        s = twell.OrthShape(rows, cols, dtype, 5, 3.0, -4.0, 2.0, 1e-7, 1.0)
        assert lib.twell_orthogonalize_workspace_size(ctypes.byref(s)) == orth_bytes(rows, cols, eb)
    for n, v, d in HEAD:
        s = ctypes.byref(twell.HeadShape(n, v, d, dtype, 8, 1.0, 0))
        assert (lib.twell_head_logprob_workspace_size(s),
                lib.twell_head_logprob_backward_workspace_size(s)) == head_bytes(n, v, d, eb)


@pytest.mark.parametrize("eb", [2, 4])
def test_what_the_gpu_tests_reach(eb):
    cuts = [orth_cuts(*s, eb) for s in BIG]
    assert all(c[0] == "big" for cut in cuts for c in cut)
    assert {cut[2][1] == 1 for cut in cuts} == {True, False}  # with and without slices of K
    # the workloads that these stand for take them too
    assert all(c[0] == "big" for c in orth_cuts(14336, 4096, eb))
    for shape in (*LARGE, (4096, 32768, 2048)):
        c = head_cuts(*shape, eb)
        assert all(c[k][0] == "big" for k in ("stats", "dl", "dw", "dx")), shape
        assert c["dx"][1] > 1
    mixed = [head_cuts(*s, eb) for s in MIXED]
    for k in ("dw", "dx"):
        assert any(c[k][0] == "mid" for c in mixed)
