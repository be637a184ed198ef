"""GPU parity of the norms around the layer (twell_norm_forward, twell_norm_backward) against the
CPU oracle in float64.

A row's sum of squares adds at most 2 * 8 terms a lane, then 6 lane steps and 16 waves, so it
carries under 40 roundings of 2^-24 each; a root, a quotient and the products behind it under 10
more.  So every float32 value is within 2^-18 (64 roundings) of the sum of the magnitudes that
were added for it, and a result in bfloat16 half a step (2^-8) of itself further.  Column sums add
the rows of a group in a chain (under 24 here), 4 groups of a workgroup, and at most 512
workgroups in 64 streams: under 64 roundings more, another 2^-18."""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import as_f64, say
from oracle.train_oracle import norm, norm_grad

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
REL = 2.0 ** -18
ALL = dict(post=True, gate=True, pre=True, y=True, dr=True)
EPS = float(np.float32(1e-5))


def make(seed, n, d, dtype, post=True, gate=True, pre=True, y=True, dr=True, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    rows = lambda: (torch.randn((n, d), generator=g)
                    * torch.exp(spread * torch.randn((n, 1), generator=g))).to(dtype)
    w = lambda: torch.randn(d, generator=g) * 0.5 + 0.7
    return dict(residual=rows(), y=rows() if y else None, w_post=w() if post else None,
                gate=w() if gate else None, w_pre=w() if pre else None,
                dr=rows() if dr else None, dx=rows() if pre else None)


def f64(t):
    return None if t is None else as_f64(t)


def cuda(t):
    return None if t is None else t.cuda()


def near(name, got, ref, of, dtype=torch.float32, rel=REL):
    step = torch.finfo(dtype).eps / 2 if dtype != torch.float32 else 0.0
    off = np.abs(as_f64(got) - ref)
    tol = rel * of + step * np.abs(ref) * (1 + 2.0 ** -8) + 1e-37
    assert np.all(off <= tol), (name, float((off / tol).max()))


def run_forward(m, alpha, eps=EPS, out=None):
    return twell.twell_norm_forward(cuda(m["residual"]), cuda(m["y"]), w_post=cuda(m["w_post"]),
                                    gate=cuda(m["gate"]), w_pre=cuda(m["w_pre"]),
                                    residual_scale=alpha, eps=eps, out=out)


def check_forward(got, m, alpha, eps=EPS):
    dt = m["residual"].dtype
    a = float(np.float32(alpha))
    r, x = norm(f64(m["residual"]), f64(m["y"]), f64(m["w_post"]), f64(m["gate"]), f64(m["w_pre"]),
                a, eps)
    of = np.abs(a * f64(m["residual"])) + np.abs(r - a * f64(m["residual"]))
    if m["y"] is not None:
        near("residual", got.residual, r, of, dt)
    if x is not None:
        std = 1 / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps)
        near("x", got.x, x, (of * std + np.abs(r * std)) * np.abs(f64(m["w_pre"])), dt)


SIZES = [(1, 8), (3, 16), (5, 504), (70, 512), (9, 520), (7, 1024), (4, 1032), (13, 2048),
         (6, 2056), (5, 4096), (3, 4104), (5, 8192), (2, 8200), (3, 16384), (4097, 8), (300, 136)]


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,d", SIZES)
def test_forward(n, d, dtype):
    say(f"norm forward {dtype} n={n} d={d}")
    m = make(n + d, n, d, dtype)
    got = run_forward(m, 0.7)
    torch.cuda.synchronize()
    check_forward(got, m, 0.7)


FORMS = [dict(ALL, gate=False), dict(ALL, post=False), dict(ALL, pre=False),
         dict(ALL, post=False, gate=False), dict(ALL, post=False, gate=False, pre=False),
         dict(ALL, post=False, pre=False), dict(ALL, gate=False, pre=False),
         dict(ALL, post=False, gate=False, y=False), dict(ALL, dr=False),
         dict(ALL, post=False, gate=False, y=False, dr=False)]


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("n,d", [(37, 256), (21, 2048), (6, 12288)])
def test_forms(n, d, form, dtype):
    """Every choice of what is given, forward and backward, several rows a group."""
    say(f"norm {dtype} {n}x{d} {form}")
    m = make(n, n, d, dtype, **form)
    alpha = 0.8 if form["y"] else 1.0
    check_forward(run_forward(m, alpha), m, alpha)
    check_backward(m, alpha)


def check_backward(m, alpha, eps=EPS, rel=REL, out=None):
    dt = m["residual"].dtype
    rout = m["residual"]  # any rows will do for the stored sum
    got = twell.twell_norm_backward(cuda(rout), cuda(m["y"]), cuda(m["dr"]), cuda(m["dx"]),
                                    w_post=cuda(m["w_post"]), gate=cuda(m["gate"]),
                                    w_pre=cuda(m["w_pre"]), residual_scale=alpha, eps=eps, out=out)
    torch.cuda.synchronize()
    ref = norm_grad(f64(rout), f64(m["y"]), f64(m["w_post"]), f64(m["gate"]), f64(m["w_pre"]),
                    f64(m["dr"]), f64(m["dx"]), float(np.float32(alpha)), eps)
    for name in ("d_residual", "dy", "dw_post", "dgate", "dw_pre"):
        if name not in ref:
            assert getattr(got, name) is None
            continue
        rows = name in ("d_residual", "dy")
        # dy's and the weights' sums carry G's own error beside theirs
        near(name, getattr(got, name), ref[name], ref["of_" + name], dt if rows else torch.float32,
             rel if name == "d_residual" else 2 * rel)
    return got


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,d", SIZES + [(9000, 64), (2100, 2048), (1100, 6144), (600, 9000)])
def test_backward(n, d, dtype):
    say(f"norm backward {dtype} n={n} d={d}")
    check_backward(make(n + d, n, d, dtype), 0.7)


@pytest.mark.gpu
@BOTH
def test_rows_of_zeros_and_of_extremes(dtype):
    """Zero rows stay zero under eps; a NaN or an infinity stays in its own row of the outputs."""
    m = make(1, 8, 256, dtype)
    for k in ("residual", "y"):
        m[k][2] = 0
    m["residual"][3] *= 1e15
    m["y"][3] *= 1e-15
    good = run_forward(m, 1.0)
    check_forward(good, m, 1.0)
    check_backward(m, 1.0)
    m["y"][5, 7] = float("nan")
    m["residual"][6, 0] = float("inf")
    bad = run_forward(m, 1.0)
    keep = [0, 1, 2, 3, 4, 7]
    assert torch.equal(bad.x[keep], good.x[keep]) and torch.equal(bad.residual[keep],
                                                                  good.residual[keep])
    assert torch.isnan(bad.x[5]).all() and torch.isnan(bad.x[6]).any()


@pytest.mark.gpu
@BOTH
def test_in_place(dtype):
    m = make(2, 50, 4096, dtype)
    ref = run_forward(m, 0.9)
    r, y = m["residual"].cuda(), m["y"].cuda()
    w = {k: cuda(m[k]) for k in ("w_post", "gate", "w_pre")}
    got = twell.twell_norm_forward(r, y, **w, residual_scale=0.9, eps=EPS,
                                   out=twell.NormOut(r, y))
    assert torch.equal(got.residual, ref.residual) and torch.equal(got.x, ref.x)
    rout, y, dr, dx = (cuda(m[k]) for k in ("residual", "y", "dr", "dx"))
    f = lambda: torch.empty(4096, device="cuda")
    ref = twell.twell_norm_backward(rout, y, dr, dx, **w, eps=EPS)
    keep = [t.clone() for t in (ref.d_residual, ref.dy, ref.dw_post, ref.dgate, ref.dw_pre)]
    got = twell.twell_norm_backward(rout, y, dr, dx, **w, eps=EPS,
                                    out=twell.NormGrads(dr, dx, f(), f(), f()))
    for a, b in zip(keep, (got.d_residual, got.dy, got.dw_post, got.dgate, got.dw_pre)):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_no_rows():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, device="cuda")
    assert twell.twell_norm_forward(e, e, w_post=w, w_pre=w).x.shape == (0, 64)
    full = lambda: torch.full((64,), 7.0, device="cuda")
    got = twell.twell_norm_backward(e, e, e, e, w_post=w, gate=w, w_pre=w,
                                    out=twell.NormGrads(e, e, full(), full(), full()))
    for t in (got.dw_post, got.dgate, got.dw_pre):
        assert not t.any()


@pytest.mark.gpu
@BOTH
def test_replayed_and_on_another_stream(dtype):
    m = make(4, 300, 1000, dtype)
    d = {k: cuda(v) for k, v in m.items()}
    w = {k: d[k] for k in ("w_post", "gate", "w_pre")}
    ws = twell.norm_backward_workspace(300, 1000, dtype, "cuda")
    call = lambda fo, go: (twell.twell_norm_forward(d["residual"], d["y"], **w, out=fo),
                           twell.twell_norm_backward(d["residual"], d["y"], d["dr"], d["dx"], **w,
                                                     out=go, workspace=ws))
    fo, go = call(None, None)
    flat = lambda: [t.clone() for o in (fo, go) for t in vars(o).values()]
    ref = flat()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(fo, go)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, flat()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(fo, go)
    for _ in range(3):
        for o in (fo, go):
            for t in vars(o).values():
                t.fill_(3)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, flat()))


# ------------------------------------------------------------------ refusals (host only)
P = 4096  # an aligned address that no call below reads


def norm_codes(n=4, d=64, dtype=1, alpha=1.0, eps=1e-6, p=(P,) * 8):
    s = twell.NormShape(n, d, dtype, alpha, eps)
    return twell.load().twell_norm_forward(ctypes.byref(s), *p, None)


no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake device pointers are passed only on a GPU-less host")


def test_refused_shapes():
    bad, un = twell.TWELL_ERR_INVALID_ARG, twell.TWELL_ERR_UNSUPPORTED
    assert norm_codes(n=0) == twell.TWELL_OK
    for kw in (dict(n=-1), dict(n=1 << 31), dict(d=0), dict(d=12), dict(dtype=2),
               dict(alpha=float("nan")), dict(alpha=float("inf")), dict(eps=0.0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf"))):
        assert norm_codes(**kw) == bad, kw
    assert norm_codes(d=16392) == un and norm_codes(n=0, d=16384) == twell.TWELL_OK
    lib = twell.load()
    size = lambda *a: lib.twell_norm_backward_workspace_size(ctypes.byref(twell.NormShape(*a)))
    assert size(0, 64, 1, 1.0, 1e-6) == 0 == size(4, 64, 1, 1.0, 0.0) == size(4, 16392, 1, 1.0, 1.0)
    # a workgroup takes four narrow rows, and writes both sums of their columns
    assert size(4, 64, 1, 1.0, 1e-6) == 2 * 64 * 4 and size(5, 64, 1, 1.0, 1e-6) == 4 * 64 * 4
    assert lib.twell_norm_forward(None, *(P,) * 8, None) == bad


@no_gpu_only
def test_refused_pointers():
    """residual, y, w_post, gate, w_pre, residual_out, x."""
    bad = twell.TWELL_ERR_INVALID_ARG
    ok = dict(residual=P, y=P, w_post=P, gate=P, w_pre=P, residual_out=P, x=P)

    def code(alpha=1.0, **kw):
        s = twell.NormShape(4, 64, 1, alpha, 1e-6)
        return twell.load().twell_norm_forward(ctypes.byref(s), *{**ok, **kw}.values(), None)

    for k in ("residual", "w_pre", "x", "residual_out", "y"):
        assert code(**{k: None}) == bad, k
    for k in ok:
        assert code(**{k: P + 8}) == bad, k
    only = dict(y=None, residual_out=None, w_post=None, gate=None)
    for kw in (dict(only, w_post=P), dict(only, gate=P), dict(only, w_pre=None, x=None),
               dict(only, alpha=0.5)):
        assert code(**kw) == bad, kw
    grad_ok = dict(residual_out=P, y=P, w_post=P, gate=P, w_pre=P, d_residual_out=P, dx=P,
                   d_residual=P, dy=P, dw_post=P, dgate=P, dw_pre=P, workspace=P)

    def grad(n=4, size=1 << 20, alpha=1.0, **kw):
        s = twell.NormShape(n, 64, 1, alpha, 1e-6)
        return twell.load().twell_norm_backward(ctypes.byref(s), *{**grad_ok, **kw}.values(), size,
                                                None)

    for k in grad_ok:
        if k != "d_residual_out":
            assert grad(**{k: None}) == bad, k
        assert grad(**{k: P + 4}) == bad, k
    assert grad(w_pre=None, dw_pre=None, dx=None, d_residual_out=None) == bad
    assert grad(w_pre=None, dw_pre=None) == bad
    assert grad(size=2 * 64 * 4 - 1) == twell.TWELL_ERR_WORKSPACE
    assert grad(n=0, w_post=None) == bad


def test_refused_tensors():
    t = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt)
    w = t(64, dt=torch.float32)
    call = twell.twell_norm_forward
    for bad in (lambda: call(t(4, 64), w_post=w, w_pre=w), lambda: call(t(4, 64)),
                lambda: call(t(4, 64), t(4, 64, dt=torch.float32), w_pre=w),
                lambda: call(t(4, 64), t(3, 64), w_pre=w), lambda: call(t(4, 64), w_pre=t(64)),
                lambda: call(t(4, 64), w_pre=w[:32]), lambda: call(t(4, 128)[:, :64], w_pre=w),
                lambda: call(t(4, 64, dt=torch.float16), w_pre=w),
                lambda: call(t(4, 64), w_pre=w),  # not on a GPU
                lambda: twell.twell_norm_backward(t(4, 64), None, None, None),
                lambda: twell.twell_norm_backward(t(4, 64), t(4, 64), t(4, 64), t(4, 64)),
                lambda: twell.twell_norm_backward(t(4, 64), None, None, t(4, 64), w_pre=w, gate=w)):
        with pytest.raises(ValueError):
            bad()
    big = torch.empty((1, 2 ** 32 + 128), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        call(big, w_pre=w)
