"""GPU parity of the log probabilities of given tokens (twell_logprob_forward) and their
gradient (twell_logprob_backward) against the CPU oracle.

Ids of the alternatives are equal.  Values: an exponent d = (x - m) * scale * log2(e) carries
three roundings, so a term 2^d is off by at most |d| * 2^-22 + 2^-22 of itself (the hardware's
exponential is within an ulp); terms of |d| above 40 weigh under 1e-12, and sums of up to 2^18
positive terms over 64 lanes add under 2^13 * 2^-24 of the worst kind, 2^-18 in practice: lse
and logp are within 2e-6 * (1 + |value| + |m * scale|), the entropy within 1e-5 * (1 + entropy).  A gradient element is
within 1e-5 of (|dlogp| + |dentropy| (1 + entropy)) * scale (p and log p each within 1e-5), plus
its rounding to bfloat16."""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import as_f64, say
from oracle.train_oracle import logprob, logprob_grad

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


def rows_on_gpu(x, stride):
    """x [N, V] on the GPU with rows `stride` elements apart, NaN between them."""
    n, v = x.shape
    buf = torch.full((n * stride + 64,), float("nan"), dtype=x.dtype, device="cuda")
    t = buf.as_strided((n, v), (stride, 1))
    t.copy_(x)
    return t


def make(seed, n, v, dtype, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, v), generator=g) * spread
    targets = torch.randint(0, v, (n,), generator=g)
    targets[::5] = -100
    if n > 3:
        targets[3] = v
    return x.to(dtype), targets


def check_forward(got, x, targets, scale, top):
    logp, entropy, lse, ids, tops = logprob(as_f64(x), targets.numpy(), np.float64(np.float32(scale)),
                                            top)
    np.testing.assert_array_equal(got.top_ids.cpu().numpy(), ids)
    big = np.abs(np.where(np.isfinite(as_f64(x)), as_f64(x), 0)).max(axis=1) * scale

    def near(name, a, b, tol):
        a = as_f64(a)
        b = np.where(np.abs(b) > np.finfo(np.float32).max, np.sign(b) * np.inf, b)  # as float32
        np.testing.assert_array_equal(np.isnan(a), np.isnan(b), name)
        np.testing.assert_array_equal(np.isinf(a), np.isinf(b), name)
        ok = np.isfinite(b)
        assert np.all(a[~ok & ~np.isnan(b)] == b[~ok & ~np.isnan(b)]), name
        tol = np.broadcast_to(tol, b.shape)
        off = np.abs(a - b)[ok]
        assert np.all(off <= tol[ok]), (name, float((off - tol[ok]).max()))
    with np.errstate(invalid="ignore"):
        near("lse", got.lse, lse, 2e-6 * (1 + np.abs(lse) + big))
        near("logp", got.logp, logp, 2e-6 * (1 + np.abs(logp) + big))
        near("top_logp", got.top_logp, tops, 2e-6 * (1 + np.abs(tops) + big[:, None]))
        near("entropy", got.entropy, entropy, 1e-5 * (1 + entropy))


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,v,stride,top,scale,index", [
    (1, 1, 1, 1, 1.0, torch.int64), (3, 2, 2, 2, 2.5, torch.int32), (5, 7, 9, 3, 1.0, torch.int64),
    (6, 15, 15, 5, 0.7, torch.int64), (9, 333, 333, 20, 1.0, torch.int32),
    (40, 1000, 1003, 32, 1.3, torch.int64), (7, 4099, 4100, 32, 1.0, torch.int64),
    (1, 131072, 131072, 20, 1.0, torch.int64), (3, 49999, 49999, 20, 0.5, torch.int32),
    (2, 262145, 262150, 32, 1.0, torch.int64), (5000, 130, 131, 4, 1.0, torch.int64),
    (4500, 65, 72, 0, 1.0, torch.int64), (70, 9001, 9001, 0, 3.0, torch.int64)])
def test_forward_matches_oracle(n, v, stride, top, scale, index, dtype):
    say(f"logprob {dtype} n={n} v={v} stride={stride} top={top}")
    x, t = make(n + v, n, v, dtype)
    got = twell.twell_logprob_forward(rows_on_gpu(x, stride), t.to(index).cuda(), top=top,
                                      scale=scale)
    torch.cuda.synchronize()
    check_forward(got, x, t, scale, top)


def odd_rows(v, dtype):
    """Rows that break naive kernels; a row per case."""
    g = torch.Generator().manual_seed(v)
    base = torch.randn((16, v), generator=g)
    low = torch.finfo(dtype).min
    x = base.to(dtype).float()
    x[0] = -torch.inf                              # nothing left
    x[1] = low                                     # a finite mask everywhere: uniform
    x[2] = -torch.inf
    x[2, v // 2] = 1.5                             # one place left
    x[3, : v - 3] = low                            # three places of weight
    x[4, ::2] = -torch.inf
    x[5] = 0.0
    x[5, ::3] = -0.0                               # all equal: the lowest columns
    x[6] = torch.arange(v) / v * 30                # rising: every batch has new maxima
    x[7] = 30 - torch.arange(v) / v * 30           # falling
    x[8] = 300.0                                   # far from zero
    x[8, 5] = 290.0
    x[9, v - 1] = 100.0                            # all the weight on the last place
    x[10, 0] = 100.0
    x[11] = -1000.0
    x[12] = torch.randint(0, 3, (v,), generator=g).float()  # many ties at the top
    x[13, 1] = float("nan")
    x[14, v - 2] = torch.inf
    x[15] = low
    x[15, 4] = -torch.finfo(dtype).min             # the widest range
    t = torch.arange(16) % v
    t[2] = v // 2
    t[9] = v - 1
    t[4] = 0                                       # a masked target
    t[11] = -1
    return x.to(dtype), t


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("v", [33, 1000, 9001, 70000])
def test_forward_odd_rows(v, dtype):
    say(f"logprob odd rows {dtype} v={v}")
    x, t = odd_rows(v, dtype)
    got = twell.twell_logprob_forward(rows_on_gpu(x, v + 1), t.cuda(), top=20)
    torch.cuda.synchronize()
    check_forward(got, x, t, 1.0, 20)
    # and one row to a wave: many copies
    many = x.repeat(300, 1)
    got = twell.twell_logprob_forward(many.cuda(), t.repeat(300).cuda(), top=20)
    torch.cuda.synchronize()
    first = twell.LogProbs(*(getattr(got, f)[-16:] for f in ("logp", "entropy", "lse", "top_ids",
                                                            "top_logp")))
    check_forward(first, x, t, 1.0, 20)


def run_backward(x, t, scale, dlogp, dent, stride=None, out_stride=None, inplace=False):
    n, v = x.shape
    xg = rows_on_gpu(x, stride or v)
    f = twell.twell_logprob_forward(xg, t.cuda(), scale=scale)
    out = xg if inplace else rows_on_gpu(torch.full_like(x, 7), out_stride or v)
    got = twell.twell_logprob_backward(xg, t.cuda(), f.lse, f.entropy, dlogp.cuda(),
                                       None if dent is None else dent.cuda(), scale=scale, out=out)
    torch.cuda.synchronize()
    return f, as_f64(got)


def check_backward(got, x, t, scale, dlogp, dent, entropy):
    s = np.float64(np.float32(scale))
    w = np.zeros(len(t)) if dent is None else as_f64(dent)
    ref = logprob_grad(as_f64(x), t.numpy(), s, as_f64(dlogp), w)
    size = (np.abs(as_f64(dlogp)) + np.abs(w) * (1 + np.nan_to_num(entropy))) * s
    tol = 1e-5 * size[:, None] + (2.0 ** -8 if x.dtype == torch.bfloat16 else 0) * np.abs(ref)
    off = np.abs(got - ref) - tol
    assert np.all(off <= 0), float(off.max())


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,v,stride,out_stride,scale,ent,inplace", [
    (1, 1, 1, 1, 1.0, True, False), (5, 7, 9, 9, 2.0, True, False), (40, 1000, 1000, 1000, 1.0, False, True),
    (33, 4099, 4099, 4099, 0.7, True, True), (9, 9001, 9001, 9008, 1.0, True, False),
    (3, 49999, 50000, 50008, 1.3, False, False), (2, 131072, 131072, 131072, 1.0, True, False)])
def test_backward_matches_oracle(n, v, stride, out_stride, scale, ent, inplace, dtype):
    say(f"logprob grad {dtype} n={n} v={v} {stride}/{out_stride}")
    x, t = make(n * 3 + v, n, v, dtype)
    g = torch.Generator().manual_seed(n)
    dlogp = torch.randn(n, generator=g)
    dent = torch.randn(n, generator=g) if ent else None
    f, got = run_backward(x, t, scale, dlogp, dent, stride, out_stride, inplace)
    check_backward(got, x, t, scale, dlogp, dent, as_f64(f.entropy))


@pytest.mark.gpu
@BOTH
def test_backward_odd_rows(dtype):
    say(f"logprob grad odd rows {dtype}")
    v = 1003
    x, t = odd_rows(v, dtype)
    t[4] = 1
    keep = [r for r in range(16) if r not in (13, 14)]
    dlogp, dent = torch.linspace(-1, 2, 16), torch.linspace(1, -1, 16)
    f, got = run_backward(x, t, 1.0, dlogp, dent, v + 2, v + 2)
    assert not got[0].any() and np.isnan(got[[13, 14]]).any(axis=1).all()
    check_backward(got[keep], x[keep], t[keep], 1.0, dlogp[keep], dent[keep],
                   as_f64(f.entropy)[keep])
    assert np.isfinite(got[keep]).all()


@pytest.mark.gpu
def test_backward_against_differences():
    """Central differences of the float64 oracle along random directions."""
    say("logprob grad differences")
    n, v, scale, eps = 6, 300, 1.3, 1e-6
    x, t = make(5, n, v, torch.float32, 1.5)
    g = torch.Generator().manual_seed(3)
    dlogp, dent = torch.randn(n, generator=g), torch.randn(n, generator=g)
    _, got = run_backward(x, t, scale, dlogp, dent)
    s = np.float64(np.float32(scale))

    def loss(y):
        logp, entropy, *_ = logprob(y, t.numpy(), s, 0)
        return (logp * as_f64(dlogp) + entropy * as_f64(dent)).sum()
    rng = np.random.default_rng(1)
    for _ in range(4):
        d = rng.standard_normal((n, v))
        fd = (loss(as_f64(x) + eps * d) - loss(as_f64(x) - eps * d)) / (2 * eps)
        assert abs(fd - (got * d).sum()) <= 1e-4 * np.linalg.norm(got) * np.sqrt(v)


@pytest.mark.gpu
def test_parts_of_longer_arrays():
    """Targets and per-row arrays that start anywhere in their own arrays."""
    say("logprob unaligned rows")
    x, t = make(9, 50, 3000, torch.bfloat16)
    x, t = x.cuda(), torch.cat([t[:1], t]).cuda()[1:]
    ref = twell.twell_logprob_forward(x, t.clone(), top=3)
    shift = lambda a: torch.cat([a.reshape(-1)[:1], a.reshape(-1)])[1:].view(a.shape)
    out = twell.LogProbs(*(shift(getattr(ref, f)).zero_() for f in (
        "logp", "entropy", "lse", "top_ids", "top_logp")))
    twell.twell_logprob_forward(x, t, top=3, out=out)
    g = shift(torch.linspace(-1, 1, 50, device="cuda"))
    d = twell.twell_logprob_backward(x, t, out.lse, out.entropy, g, g)
    dref = twell.twell_logprob_backward(x, t.clone(), ref.lse, ref.entropy, g.clone(), g.clone())
    torch.cuda.synchronize()
    for f in ("logp", "entropy", "lse", "top_ids", "top_logp"):
        assert torch.equal(getattr(out, f), getattr(ref, f))
    assert torch.equal(d, dref)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """More than 2^31 logits: the last row is scored and differentiated."""
    say("logprob offsets past 2^31")
    v, n = 262144, 8300
    x = torch.zeros((n, v), dtype=torch.bfloat16, device="cuda")
    x[n - 1, v - 1] = 20.0
    t = torch.full((n,), v - 1, dtype=torch.int64, device="cuda")
    f = twell.twell_logprob_forward(x, t, top=2)
    d = twell.twell_logprob_backward(x, t, f.lse, None, torch.ones(n, device="cuda"), out=x)
    torch.cuda.synchronize()
    ref = 20.0 - np.log(np.exp(20.0) + v - 1)
    assert abs(float(f.logp[n - 1]) - ref) < 1e-5
    assert abs(float(f.logp[n - 2]) + np.log(v)) < 4e-5
    assert f.top_ids[n - 1].tolist() == [v - 1, 0] and f.top_ids[n - 2].tolist() == [0, 1]
    assert abs(float(d[n - 1, v - 1]) - (1 - np.exp(ref))) < 1e-5


@pytest.mark.gpu
def test_zero_rows_graph_and_side_stream():
    say("logprob n=0, graph, side stream")
    e = twell.twell_logprob_forward(torch.empty((0, 50), device="cuda"),
                                    torch.empty((0,), dtype=torch.int64, device="cuda"), top=3)
    assert e.logp.shape == (0,) and e.top_ids.shape == (0, 3)
    for n, v in ((20, 20000), (4200, 500)):
        x, t = make(1, n, v, torch.bfloat16)
        x, t = x.cuda(), t.cuda()
        ws = twell.logprob_workspace(n, v, 5, x.dtype, "cuda")
        ref = twell.twell_logprob_forward(x, t, top=5)
        g = torch.ones(n, device="cuda")
        dref = twell.twell_logprob_backward(x, t, ref.lse, ref.entropy, g, g)
        out, dout = twell.LogProbs.empty(n, 5, "cuda"), torch.empty_like(x)

        def both():
            twell.twell_logprob_forward(x, t, top=5, out=out, workspace=ws)
            twell.twell_logprob_backward(x, t, out.lse, out.entropy, g, g, out=dout)

        def same():
            return all(torch.equal(getattr(out, f), getattr(ref, f)) for f in
                       ("logp", "entropy", "lse", "top_ids", "top_logp")) and torch.equal(dout, dref)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            both()
        side.synchronize()
        assert same()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            both()
        for _ in range(3):
            out.logp.fill_(7)
            out.top_ids.fill_(7)
            dout.fill_(7)
            ws.fill_(255)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert same()


@pytest.mark.gpu
def test_refusals():
    x = torch.zeros((4, 64), device="cuda")
    t = torch.zeros((4,), dtype=torch.int64, device="cuda")
    z = torch.zeros((4,), device="cuda")
    fwd, bwd = twell.twell_logprob_forward, twell.twell_logprob_backward
    with pytest.raises(ValueError, match="int32 or int64"):
        fwd(x, t.short())
    with pytest.raises(ValueError, match="not supported"):
        fwd(x.double(), t)
    with pytest.raises(ValueError, match="contiguous rows"):
        fwd(x.t().contiguous().t(), t)
    with pytest.raises(ValueError, match="targets must have shape"):
        fwd(x, t[:3])
    with pytest.raises(ValueError, match="needs the forward's entropy"):
        bwd(x, t, z, None, z, z)
    with pytest.raises(ValueError, match="out must"):
        bwd(x, t, z, None, z, out=x.bfloat16())
    for kw in (dict(top=33), dict(top=-1), dict(scale=0.0), dict(scale=float("inf"))):
        with pytest.raises(twell.TwellError) as e:
            fwd(x, t, **kw)
        assert e.value.code == twell.TWELL_ERR_INVALID_ARG
    with pytest.raises(twell.TwellError) as e:
        fwd(x[:, :5], t, top=6)
    assert e.value.code == twell.TWELL_ERR_INVALID_ARG
    big = torch.zeros((1, 100000), device="cuda")
    with pytest.raises(twell.TwellError) as e:
        fwd(big, t[:1], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == twell.TWELL_ERR_WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="fake device pointers are passed only on a GPU-less host")
def test_host_checks():
    lib = twell.load()
    p = 4096
    bad = twell.TWELL_ERR_INVALID_ARG

    def shape(**kw):
        f = dict(n_rows=4, row_stride=64, vocab=64, dtype=1, index_bytes=8, top=2, scale=1.0,
                 reserved=0)
        return twell.LogprobShape(**{**f, **kw})

    def fwd(s, x=p, t=p, logp=p, ids=p, ws=p, wsb=0):
        return lib.twell_logprob_forward(ctypes.byref(s), x, t, logp, p, p, ids, p, ws, wsb, None)

    def bwd(s, x=p, lse=p, ent=p, de=p, d=2 * p, stride=64):
        return lib.twell_logprob_backward(ctypes.byref(s), x, p, lse, ent, p, de, d, stride, None)
    for kw in (dict(n_rows=-1), dict(row_stride=63), dict(vocab=0), dict(dtype=2),
               dict(index_bytes=1), dict(top=65), dict(top=33), dict(scale=-1.0),
               dict(scale=float("nan")), dict(reserved=1)):
        assert fwd(shape(**kw)) == bad, kw
        assert bwd(shape(**kw)) == bad, kw
        assert lib.twell_logprob_workspace_size(ctypes.byref(shape(**kw))) == 0
    assert fwd(shape(n_rows=1 << 27)) == twell.TWELL_ERR_UNSUPPORTED
    assert fwd(shape(), x=None) == bad and fwd(shape(), ids=None) == bad
    assert fwd(shape(), x=p + 8) == bad and fwd(shape(), logp=p + 2) == bad
    assert fwd(shape(), t=p + 4) == bad
    s = shape(vocab=100000, row_stride=100000)
    need = lib.twell_logprob_workspace_size(ctypes.byref(s))
    assert need > 0 and fwd(s, ws=None, wsb=need) == bad
    assert fwd(s, wsb=need - 1) == twell.TWELL_ERR_WORKSPACE
    assert bwd(shape(), lse=None) == bad and bwd(shape(), ent=None) == bad
    assert bwd(shape(), stride=63) == bad and bwd(shape(), d=p + 8) == bad
    assert bwd(shape(row_stride=72), d=p, stride=64) == bad  # in place with another stride
    empty = shape(n_rows=0)
    assert fwd(empty) == twell.TWELL_OK and bwd(empty) == twell.TWELL_OK
