"""GPU parity of the output head's log probabilities without logits (twell_head_logprob_forward)
and their gradient (twell_head_logprob_backward) against the CPU oracle in float64.

A logit z is a float32 sum of d products (float32 operands: of 3 d products of half-precision
parts).  MFMA cuts it a few times per 16 products, under 1.5 d times in all; partial sums of terms
of random sign stay within 4 times the root a of the summed squares, and independent roundings
(2^-24 each) add up as their root: within six deviations that is ez = 24 sqrt(1.5 d) a 2^-24.  The
parts' own errors, 2^-22.4 of a term in the mean square at most, and the cuts' one-sided mean,
d / 16 * 2^-24 of z, stay under that for the d here.  lse and logp carry the row's largest ez, and 2^-20 (1 + |lse|) from
the exponentials, sums and the logarithm.  dl = g (1 - p) is off by |g| p (2 ez + 2^-20), with
bfloat16 operands by half a step of itself more; dx and dw by those errors through the product,
their own float32 sum (ez with K for d) and half a step of the result."""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import as_f64, say
from oracle.train_oracle import head_logprob, head_logprob_grad

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
U = 2.0 ** -24


def make(seed, n, v, d, dtype, scale=1.0, index=torch.int64):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn((v, d), generator=g) * 2 * d ** -0.5).to(dtype)
    t = torch.randint(0, v, (n,), generator=g)
    x = (torch.randn((n, d), generator=g) + torch.rand((n, 1), generator=g) * w[t].float()).to(dtype)
    t[1::5] = -100
    if n > 3:
        t[3] = v
    return dict(x=x, w=w, t=t.to(index), scale=scale,
                dlogp=-torch.rand(n, generator=g) / n)


def root_sum(a, b):
    """sqrt of (a^2) (b^2)^T: the root of each sum's squared terms."""
    return np.sqrt((a * a) @ (b * b).T)


def errors_of_z(x, w, scale):
    d = x.shape[1]
    return scale * (24 * np.sqrt(1.5 * d) * U) * root_sum(x, w)


def forward(m, **kw):
    return twell.twell_head_logprob_forward(m["x"].cuda(), m["w"].cuda(), m["t"].cuda(),
                                            scale=m["scale"], **kw)


def backward(m, stats, **kw):
    return twell.twell_head_logprob_backward(m["x"].cuda(), m["w"].cuda(), m["t"].cuda(), stats,
                                             m["dlogp"].cuda(), scale=m["scale"], **kw)


def within(name, got, ref, tol):
    off = np.abs(as_f64(got) - ref)
    assert np.all(off <= tol), (name, float((off / np.maximum(tol, 1e-300)).max()))


def check(m):
    x, w, t = as_f64(m["x"]), as_f64(m["w"]), m["t"].numpy()
    scale = float(np.float32(m["scale"]))
    step = torch.finfo(m["x"].dtype).eps / 2
    part = step if m["x"].dtype == torch.bfloat16 else 0.0  # dl's own rounding
    logp, lse, stats, z = head_logprob(x, w, t, scale)
    ez = errors_of_z(x, w, scale)
    e_row = ez.max(axis=1)
    got = forward(m)
    torch.cuda.synchronize()
    tol = 2 * e_row + 2.0 ** -20 * (1 + np.abs(lse))
    within("lse", got.lse, lse, tol)
    within("logp", got.logp, logp, tol)
    assert not got.logp[(m["t"] < 0) | (m["t"] >= len(w))].any()
    within("max", got.stats[:, 0], stats[:, 0], e_row)
    within("sum", got.stats[:, 1], stats[:, 1], stats[:, 1] * (2 * tol))
    grads = backward(m, got.stats)
    torch.cuda.synchronize()
    dlogp = as_f64(m["dlogp"])
    dx, dw, dl = head_logprob_grad(x, w, t, dlogp, scale)
    ok = (t >= 0) & (t < len(w))
    g = np.where(ok, np.abs(dlogp) * scale, 0.0)
    p = np.exp(z - lse[:, None])
    e_dl = g[:, None] * p * (2 * e_row[:, None] + 2.0 ** -20) + np.abs(dl) * (part + 2 * U)
    xm = np.where(ok[:, None], x, 0.0)
    sums = lambda k: 24 * np.sqrt(1.5 * k) * U
    for name, a, ref, b, e in (("dx", grads.dx, dx, w.T, e_dl), ("dw", grads.dw, dw, xm.T, e_dl.T)):
        d0 = dl if name == "dx" else dl.T
        within(name, a, ref, e @ np.abs(b.T) + sums(len(b.T)) * root_sum(d0, b)
               + step * np.abs(ref) * 1.01 + 1e-37)
    assert not grads.dx[torch.from_numpy(~ok)].any()
    return got, grads


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,v,d,scale,index", [
    (1, 1, 8, 1.0, torch.int64), (1, 500, 64, 1.0, torch.int32), (2, 63, 16, 2.0, torch.int64),
    (3, 129, 72, 1.0, torch.int64), (17, 1000, 128, 0.7, torch.int64),
    (32, 513, 320, 1.0, torch.int64), (33, 257, 200, 1.0, torch.int32),
    (64, 4099, 64, 1.0, torch.int64), (65, 300, 1032, 1.5, torch.int64),
    (130, 2000, 256, 1.0, torch.int64), (300, 777, 520, 1.0, torch.int64),
    (1000, 2900, 64, 1.0, torch.int64), (5, 20000, 24, 1.0, torch.int64),
    (3000, 4100, 64, 1.0, torch.int64), (4090, 5000, 40, 1.0, torch.int64),
    (257, 3, 2048, 1.0, torch.int64), (16, 4096, 136, 1.0, torch.int64),
    (17, 4097, 1000, 1.0, torch.int64), (48, 9005, 376, 0.7, torch.int64),
    (64, 300000, 96, 1.0, torch.int64), (2, 150000, 184, 1.0, torch.int32),
    (70, 70000, 8, 1.0, torch.int64)])
def test_matches_oracle(n, v, d, scale, index, dtype):
    say(f"head {dtype} n={n} v={v} d={d} scale={scale}")
    check(make(n + v + d, n, v, d, dtype, scale, index))


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,v,d", [(20, 60000, 1000), (70, 100000, 1344), (1100, 100000, 64)])
def test_vocabularies_of_several_pieces(n, v, d, dtype):
    say(f"head in pieces {dtype} n={n} v={v} d={d}")
    check(make(n + v + d, n, v, d, dtype))


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n", [1, 40, 70, 200])
def test_every_bit_of_the_operands(n, dtype):
    """One product a logit: x and w one-hot rows with values of all mantissa bits.  bfloat16: z is
    exact (16 bits).  float32: x and w are hi + lo within 2^-23 each, the product lo lo, left out,
    is at most 2^-22 of z, and adding hi hi to the two small products cuts at most 2^-23 of z (adding
    those two 2^-10 of that): (2 + 2 + 1.001) 2^-23 = 10.1 * 2^-24 in all."""
    d, v = 64, 192
    g = torch.Generator().manual_seed(n)
    x, w = torch.zeros((n, d)), torch.zeros((v, d))
    at = torch.randint(0, d, (n,), generator=g)
    x[torch.arange(n), at] = 1 + torch.rand(n, generator=g)
    w[torch.arange(v), torch.arange(v) % d] = 2 + torch.rand(v, generator=g)
    m = dict(x=x.to(dtype), w=w.to(dtype), t=torch.arange(n) % v, scale=1.0,
             dlogp=torch.ones(n))
    got = forward(m)
    z = as_f64(m["x"]) @ as_f64(m["w"]).T
    within("max", got.stats[:, 0], z.max(axis=1),
           (10.1 * U if dtype == torch.float32 else 0) * z.max(axis=1))


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,v,d", [(5, 300, 64), (70, 1000, 72), (200, 400, 64)])
def test_masked_rows_spread_nothing(n, v, d, dtype):
    """Rows without a target may hold NaN and infinities; so may their dlogp."""
    m = make(n, n, v, d, dtype)
    clean, grads = check(m)
    skip = (m["t"] < 0) | (m["t"] >= v)
    m["x"][skip] = float("nan")
    m["x"][3] = float("inf")
    m["dlogp"][skip] = float("nan")
    got = forward(m)
    again = backward(m, got.stats)
    assert not got.logp[skip].any() and torch.equal(got.logp, clean.logp)
    assert torch.equal(again.dx, grads.dx) and torch.equal(again.dw, grads.dw)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n", [5, 200])
def test_masked_rows_beside_infinite_weights(n, dtype):
    """A row without a target has no gradient, also where w holds infinities and NaN."""
    m = make(3, n, 300, 64, dtype)
    m["w"][7, 5] = float("inf")
    m["w"][8, 6] = float("nan")
    got = forward(m)
    grads = backward(m, got.stats)
    skip = (m["t"] < 0) | (m["t"] >= 300)
    assert not got.logp[skip].any() and torch.isnan(got.logp[~skip]).all()
    assert not grads.dx[skip].any()


@pytest.mark.gpu
def test_more_elements_than_a_launch_has_lanes():
    """x and dx past 2^32 elements: rows at both ends have the results of a small call with the
    same weights, and dw is theirs."""
    say("2^20 + 72 rows of 4096")
    n, d, v = (1 << 20) + 72, 4096, 40
    part = make(4, 144, v, d, torch.bfloat16)
    part["dlogp"] = torch.full((144,), -2.0 ** -20)
    x, t = part["x"].cuda(), part["t"].cuda()
    big = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    targets = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    # the first and the last 72 rows have targets
    for rows, at in ((slice(0, 72), slice(0, 72)), (slice(n - 72, n), slice(72, 144))):
        big[rows] = x[at]
        targets[rows] = t[at]
    dlogp = torch.full((n,), -2.0 ** -20, device="cuda")
    w = part["w"].cuda()
    got = twell.twell_head_logprob_forward(big, w, targets)
    grads = twell.twell_head_logprob_backward(big, w, targets, got.stats, dlogp)
    torch.cuda.synchronize()
    small = forward(part)
    ref = backward(part, small.stats)
    ends = lambda v: torch.cat([v[:72], v[n - 72:]]).double()
    # both are within ez of z; each dl is then within a step of bfloat16 (2^-7) of the other's,
    # and sums of |dl| over a row stay under 2 |dlogp|, over a column under its terms' sizes
    ez = 2 * errors_of_z(as_f64(x), as_f64(w), 1.0).max()
    for a, b in ((got.logp, small.logp), (got.lse, small.lse)):
        assert float((ends(a) - b).abs().max()) <= 2 * ez + 2.0 ** -19 * (1 + float(b.abs().max()))
    step = 2.0 ** -7 + 4 * ez
    off = (ends(grads.dx) - ref.dx.double()).abs()
    size = 2 * dlogp[0].abs() * w.double().abs().max()
    assert bool((off <= 2.0 ** -7 * ref.dx.double().abs() + step * size).all())
    assert not got.logp[72:n - 72].any()
    assert not grads.dx[72:n - 72].any()
    off = (grads.dw.double() - ref.dw.double()).abs()
    size = dlogp[0].abs() * x.double().abs().sum(0)
    assert bool((off <= 2.0 ** -7 * ref.dw.double().abs() + step * size).all())


@pytest.mark.gpu
@BOTH
def test_rows_without_a_target_alone(dtype):
    m = make(1, 40, 500, 64, dtype)
    m["t"][:] = -1
    got = forward(m)
    grads = backward(m, got.stats)
    assert not got.logp.any() and torch.isfinite(got.lse).all()
    assert not grads.dx.any() and not grads.dw.any()


@pytest.mark.gpu
@BOTH
def test_nan_and_infinities(dtype):
    """A NaN row is NaN and leaves the other rows alone; a column of z = -inf has no weight."""
    m = make(9, 20, 300, 64, dtype)
    m["t"] = torch.arange(20) * 7
    good = forward(m)
    m["x"][4, 3] = float("nan")
    got = forward(m)
    assert torch.isnan(got.logp[4]) and torch.isnan(got.lse[4])
    keep = torch.arange(20) != 4
    assert torch.equal(got.logp[keep], good.logp[keep])
    if dtype == torch.bfloat16:
        m = make(9, 20, 300, 64, dtype)
        m["t"] = torch.arange(20) * 7
        m["x"][:, 0] = 1
        m["w"][299] = 0
        m["w"][299, 0] = -float("inf")
        m["w"][:299, 0] = 0
        x, w = as_f64(m["x"]), as_f64(m["w"])
        got = forward(m)
        ref = head_logprob(x, w[:299], m["t"].numpy(), 1.0)
        within("logp", got.logp, ref[0], 1e-4)
        grads = backward(m, got.stats)
        assert not grads.dw[299].any()
        # every column so: nothing is left
        m["w"][:] = 0
        m["w"][:, 0] = -float("inf")
        got = forward(m)
        assert torch.isneginf(got.logp).all() and torch.isneginf(got.lse).all()
        assert not backward(m, got.stats).dw.any()


@pytest.mark.gpu
@BOTH
def test_logits_of_hundreds(dtype):
    """Rows whose logits are far from zero keep their probabilities: the gradient takes the
    maximum and the sum, not their joint logarithm."""
    n, v, d = 30, 700, 64
    m = make(3, n, v, d, dtype)
    m["w"][:, 0] = 16.0
    m["x"][:, 0] = torch.tensor([50.0, -50.0, 20.0]).repeat(10).to(dtype)
    check(m)


@pytest.mark.gpu
@BOTH
def test_gradient_against_differences(dtype):
    """(f(x + h u) - f(x - h u)) / 2h of the oracle's f along random directions, on the stored
    operands."""
    m = make(6, 12, 90, 64, dtype)
    m["t"] = torch.arange(12) * 3
    got = backward(m, forward(m).stats)
    x, w, t, c = as_f64(m["x"]), as_f64(m["w"]), m["t"].numpy(), as_f64(m["dlogp"])
    f = lambda x, w: float((c * head_logprob(x, w, t, 1.0)[0]).sum())
    rng = np.random.default_rng(0)
    rel = 2.0 ** -7 if dtype == torch.bfloat16 else 2.0 ** -17
    for name, a in (("dx", x), ("dw", w)):
        u, h = rng.normal(size=a.shape), 1e-5
        diff = ((f(x + h * u, w) - f(x - h * u, w)) if name == "dx"
                else (f(x, w + h * u) - f(x, w - h * u))) / (2 * h)
        mine = as_f64(getattr(got, name))
        assert abs((mine * u).sum() - diff) <= rel * np.sqrt(((mine * u) ** 2).sum()) * 4 + 1e-9


@pytest.mark.gpu
@BOTH
def test_no_rows(dtype):
    e = torch.empty((0, 64), dtype=dtype, device="cuda")
    w = torch.ones((100, 64), dtype=dtype, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    assert twell.twell_head_logprob_forward(e, w, t).logp.shape == (0,)
    f = torch.empty(0, device="cuda")
    out = twell.HeadGrads(e, torch.full_like(w, 7))
    twell.twell_head_logprob_backward(e, w, t, f.view(0, 2), f, out=out)
    assert not out.dw.any()


@pytest.mark.gpu
@BOTH
def test_replayed_and_on_another_stream(dtype):
    m = make(5, 90, 1500, 72, dtype)
    x, w, t, c = m["x"].cuda(), m["w"].cuda(), m["t"].cuda(), m["dlogp"].cuda()
    wsf = twell.head_logprob_workspace(90, 1500, 72, dtype, "cuda")
    wsb = twell.head_logprob_workspace(90, 1500, 72, dtype, "cuda", backward=True)

    def call(fo, go):
        fo = twell.twell_head_logprob_forward(x, w, t, out=fo, workspace=wsf)
        return fo, twell.twell_head_logprob_backward(x, w, t, fo.stats, c, out=go, workspace=wsb)
    fo, go = call(None, None)
    flat = lambda: [a.clone() for o in (fo, go) for a in vars(o).values()]
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
            for a in vars(o).values():
                a.fill_(3)
        wsf.fill_(255)
        wsb.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref, flat()))


# ------------------------------------------------------------------ refusals (host only)
P = 4096  # an aligned address that no call below reads
OK, BAD, UNSUPPORTED = twell.TWELL_OK, twell.TWELL_ERR_INVALID_ARG, twell.TWELL_ERR_UNSUPPORTED


def codes(n=0, v=100, d=64, dtype=1, index=8, scale=1.0, reserved=0):
    s = ctypes.byref(twell.HeadShape(n, v, d, dtype, index, scale, reserved))
    lib = twell.load()
    return lib.twell_head_logprob_forward(s, *(None,) * 7, 0, None)


def test_refused_shapes():
    assert codes() == OK
    for kw in (dict(n=-1), dict(v=0), dict(d=0), dict(d=12), dict(dtype=2), dict(index=2),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(reserved=1)):
        assert codes(**kw) == BAD, kw
    for kw in (dict(n=(1 << 24) + 1), dict(v=(1 << 24) + 1), dict(d=(1 << 16) + 8),
               dict(n=1 << 20, v=(1 << 18) + 1), dict(n=(1 << 18) + 1, d=1 << 16),
               dict(v=(1 << 20) + 1, d=1 << 16)):
        assert codes(**kw) == UNSUPPORTED, kw
    lib = twell.load()
    for f in (lib.twell_head_logprob_workspace_size, lib.twell_head_logprob_backward_workspace_size):
        size = lambda **kw: f(ctypes.byref(twell.HeadShape(*{**dict(
            n=5, v=100, d=64, dtype=1, index=8, scale=1.0, reserved=0), **kw}.values())))
        assert size() > 0 == size(n=0) == size(d=4) == size(n=(1 << 24) + 1)
        # the largest shapes are counted without overflow
        assert size(n=1 << 24, v=1 << 14, d=1024) > 1 << 24
        assert size(n=1 << 14, v=1 << 24, d=4096, dtype=0) > 1 << 24
    assert lib.twell_head_logprob_forward(None, *(P,) * 7, 0, None) == BAD


no_gpu_only = pytest.mark.skipif(torch.cuda.is_available(),
                                 reason="fake device pointers are passed only on a GPU-less host")


@no_gpu_only
def test_refused_pointers():
    lib = twell.load()
    fwd = dict(x=P, w=P, targets=P, logp=P, lse=P, stats=P, workspace=P)
    bwd = dict(x=P, w=P, targets=P, stats=P, dlogp=P, dx=P, dw=P, workspace=P)
    for ok, name, odd in ((fwd, "twell_head_logprob_forward", dict(logp=2, lse=2, stats=4)),
                          (bwd, "twell_head_logprob_backward", dict(stats=4, dlogp=2))):
        def code(n=4, size=1 << 40, **kw):
            s = ctypes.byref(twell.HeadShape(n, 100, 64, 1, 8, 1.0, 0))
            return getattr(lib, name)(s, *{**ok, **kw}.values(), size, None)
        for k in ok:
            assert code(**{k: None}) == BAD, (name, k)
            assert code(**{k: P + odd.get(k, 4)}) == BAD, (name, k)
        assert code(size=64) == twell.TWELL_ERR_WORKSPACE
    assert code(n=0, dw=None) == BAD


def test_refused_tensors():
    t = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt)
    ids = torch.zeros(4, dtype=torch.int64)
    f = twell.twell_head_logprob_forward
    st, dl = t(4, 2, dt=torch.float32), t(4, dt=torch.float32)
    for bad in (lambda: f(t(4, 64), t(10, 64), ids),  # not on a GPU
                lambda: f(t(4, 64), t(10, 72), ids), lambda: f(t(4, 64), t(10, 64), ids[:3]),
                lambda: f(t(4, 64), t(10, 64, dt=torch.float32), ids),
                lambda: f(t(4, 64, dt=torch.float16), t(10, 64, dt=torch.float16), ids),
                lambda: f(t(4, 64), t(10, 64), ids.float()),
                lambda: f(t(4, 128)[:, :64], t(10, 64), ids),
                lambda: f(t(4, 64), t(64, 10).t(), ids),
                lambda: twell.twell_head_logprob_backward(t(4, 64), t(10, 64), ids, st[:3], dl),
                lambda: twell.twell_head_logprob_backward(t(4, 64), t(10, 64), ids, st, dl.double())):
        with pytest.raises(ValueError):
            bad()
    big = torch.empty((2 ** 32 + 128, 8), dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        f(torch.empty((4, 8), dtype=torch.bfloat16, device="meta"), big,
          torch.empty(4, dtype=torch.int64, device="meta"))
    with pytest.raises(ValueError, match="32 bits"):
        twell.head_logprob_workspace(1, 2 ** 32 + 1, 64, torch.bfloat16, "meta")
