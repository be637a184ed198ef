"""GPU parity of the 8-bit activation checkpoints (twell_act8_pack, twell_act8_unpack) and of
the backward pass that reads one (ffn_sparse_backward_act8) against the CPU oracle.

Codes: the quotient x * 127 / a is formed in float32.  For bfloat16 x the product is exact (15
bits) and the quotient of such integers by an 8-bit one lies at least 1/512 from any other
half-integer, so the correctly rounded quotient rounds as the real one does: codes are equal.
For float32 x the quotient (at most 127) carries two roundings of 2^-24, 1.6e-5 in all, so a code
is within 0.5 + 2e-5 of the real quotient.  Scales and read-back values are single float32
operations: equal bit for bit.

Backward: dw_down, dw_up_t and db_up are float32 sums of float32 products for both storage types
(1e-4 of max|ref|, the library's float32 bar); dx is TOL[dtype] of max|ref| as in the plain
backward.  Integer-valued layers are exact."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from activation_sparse_transformer_amd import synth, twell
from gpu_helpers import TOL, as_f32, as_f64, assert_close_rel, oracle_inputs, say, u32
from oracle.train_oracle import act8_decode, act8_quotients

F32 = TOL[torch.float32]


def wide_x(seed, n, d, dtype):
    """Rows of very different sizes, a zero block, a block of one value, signed zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, d), generator=g) * 10 ** (torch.rand((n, 1), generator=g) * 60 - 30)
    if n > 2:
        x[1] = 0
        x[2, :8] = -x[2, 0]
        x[2, 8:] = -0.0
    return x.to(dtype)


def on_gpu_pack(x):
    a = twell.twell_act8_pack(x.cuda())
    y = twell.twell_act8_unpack(a)
    torch.cuda.synchronize()
    return a, a.codes.cpu().numpy(), a.scales.cpu().numpy(), y.cpu()


def check_readback(codes, scales, y, d):
    per = np.repeat(scales, 128, axis=1)[:, :d]
    with np.errstate(invalid="ignore"):
        want = torch.from_numpy(codes[:, :d].astype(np.float32) * per).to(y.dtype)
    y, want = as_f32(y), as_f32(want)
    np.testing.assert_array_equal(np.isnan(y), np.isnan(want))  # any NaN bits
    np.testing.assert_array_equal(u32(np.nan_to_num(y)), u32(np.nan_to_num(want)))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,d", [(1, 8), (3, 128), (64, 136), (5, 1000), (300, 2048), (17, 8200),
                                 (4096, 24)])
def test_pack_matches_oracle(n, d, dtype):
    say(f"act8 pack {dtype} n={n} d={d}")
    x = wide_x(n * 7 + d, n, d, dtype)
    _, codes, scales, y = on_gpu_pack(x)
    q, a = act8_quotients(as_f64(x))
    np.testing.assert_array_equal(u32(scales), u32(a.astype(np.float32) / np.float32(127)))
    if dtype == torch.bfloat16:
        np.testing.assert_array_equal(codes[:, :d], np.rint(q).astype(np.int8))
    else:
        assert np.abs(codes[:, :d] - q).max() <= 0.5 + 2e-5
    assert not codes[:, d:].any()
    check_readback(codes, scales, y, d)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_pack_extreme_values(dtype):
    """The type's largest value, subnormals, ties, NaN and infinities: only the block that holds
    a NaN or an infinity reads back as NaN."""
    say(f"act8 extreme {dtype}")
    big = torch.finfo(dtype).max
    x = torch.zeros((7, 264), dtype=dtype)
    x[0, 0], x[0, 1], x[0, 2] = big, -big / 2, big / 256
    x[1, 130], x[1, 131] = 2.0 ** -130, -2.0 ** -131  # subnormal in both types
    x[2, 0], x[2, 1] = float("nan"), 3.0
    x[2, 200] = 5.0
    x[3, 129], x[3, 0] = -float("inf"), 1.0
    x[4] = torch.linspace(-1.0, 1.0, 264).to(dtype)
    x[5, 260], x[5, 261] = 2.0, 1.0  # a quotient of exactly 63.5: to the even 64
    x[6, 0], x[6, 1] = 2.0, -1.0
    _, codes, scales, y = on_gpu_pack(x)
    bad = np.zeros((7, 3), bool)
    bad[2, 0] = bad[3, 1] = True
    np.testing.assert_array_equal(np.isnan(scales), bad)
    columns = np.repeat(bad, 128, axis=1)[:, :264]
    np.testing.assert_array_equal(torch.isnan(y).numpy(), columns)
    assert not codes[:, :264][columns].any()
    ok = np.where(columns, 0.0, as_f64(x))
    q, a = act8_quotients(ok)
    assert np.abs(codes[:, :264] - q)[~columns].max() <= 0.5 + 2e-5
    assert codes[5, 261] == 64 and codes[6, 1] == -64
    assert torch.isfinite(y[0]).all()  # the type's largest value reads back finite
    check_readback(codes, scales, y, 264)


@pytest.mark.gpu
def test_pack_zero_rows_and_side_stream():
    say("act8 n=0, side stream")
    a = twell.twell_act8_pack(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"))
    assert twell.twell_act8_unpack(a).shape == (0, 64)
    x = wide_x(3, 500, 512, torch.float32).cuda()
    ref = twell.twell_act8_unpack(twell.twell_act8_pack(x))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = twell.twell_act8_unpack(twell.twell_act8_pack(x))
    s.synchronize()
    assert torch.equal(got, ref)


@pytest.mark.gpu
def test_pack_graph_replays():
    say("act8 graph")
    x = wide_x(9, 300, 520, torch.bfloat16).cuda()
    a = twell.twell_act8_pack(x)
    y = twell.twell_act8_unpack(a)
    torch.cuda.synchronize()
    ref = y.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        twell.twell_act8_pack(x, out=a)
        twell.twell_act8_unpack(a, out=y)
    for _ in range(3):
        y.fill_(7)
        a.codes.fill_(1)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref)


@pytest.mark.gpu
def test_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        twell.twell_act8_pack(torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")[:, :64])
    with pytest.raises(ValueError, match="not supported"):
        twell.twell_act8_pack(x.half())
    with pytest.raises(ValueError, match="out holds"):
        twell.twell_act8_pack(x, out=twell.Act8.empty(5, 64, torch.bfloat16, "cuda:0"))
    with pytest.raises(twell.TwellError) as e:
        twell.twell_act8_pack(torch.zeros((4, 60), dtype=torch.bfloat16, device="cuda"))
    assert e.value.code == twell.TWELL_ERR_INVALID_ARG
    a = twell.twell_act8_pack(x)
    a.scales = a.scales.cpu()
    with pytest.raises(ValueError, match="scales"):
        twell.twell_act8_unpack(a)


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="fake device pointers are passed only on a GPU-less host")
def test_host_checks():
    lib = twell.load()
    p = 4096
    call = lambda n, d, dt, x, a: (
        lib.twell_act8_pack(n, d, dt, x, ctypes.byref(a) if a else None, None),
        lib.twell_act8_unpack(n, d, dt, ctypes.byref(a) if a else None, x, None))
    ok = twell.Act8Struct(p, p)
    bad = (twell.TWELL_ERR_INVALID_ARG,) * 2
    assert call(4, 12, 1, p, ok) == bad          # d_model not a multiple of 8
    assert call(-1, 64, 1, p, ok) == bad
    assert call(4, 64, 2, p, ok) == bad          # dtype
    assert call(4, 64, 1, None, ok) == bad
    assert call(4, 64, 1, p + 4, ok) == bad      # misaligned
    assert call(4, 64, 1, p, None) == bad
    assert call(4, 64, 1, p, twell.Act8Struct(p, None)) == bad
    assert call(4, 64, 1, p, twell.Act8Struct(p + 8, p)) == bad
    assert call(1 << 28, 256, 1, p, ok) == (twell.TWELL_ERR_UNSUPPORTED,) * 2
    assert call(0, 64, 1, None, twell.Act8Struct(None, None)) == (twell.TWELL_OK,) * 2


# ------------------------------------------------------------------ backward
def layer(n, dm, dff, dtype, b0, seed):
    cfg = synth.FfnConfig("act8", n, dm, dff, 64, 4, dtype, b0, token_scale_var=0.5, seed=seed)
    t = synth.make_inputs(cfg)
    t["dy"] = synth.make_grad(cfg)
    return cfg, t


def run_backward(t, x8, h, T, C, dense_capacity=None):
    d = {k: v.cuda() for k, v in t.items()}
    hy, status = twell.twell_pack(h.cuda(), T, C, dense_capacity=dense_capacity)
    g = twell.ffn_sparse_backward_act8(x8, d["w_up_t"], d["w_down"], hy, d["dy"])
    torch.cuda.synchronize()
    return hy, int(status.item()), g


def check(g, ref, dtype):
    assert_close_rel(as_f64(g.dw_down), ref.dw_down, F32, "dw_down")
    assert_close_rel(as_f64(g.dw_up_t), ref.dw_up_t, F32, "dw_up_t")
    assert_close_rel(as_f64(g.db_up), ref.db, F32, "db_up")
    assert_close_rel(as_f64(g.dx), ref.dx, TOL[dtype], "dx")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,dm,dff,T,C,b0", [
    (1, 128, 512, 64, 4, -1.645),
    (40, 136, 768, 128, 4, -1.645),     # one slice, a last half vector
    (300, 256, 1024, 64, 4, -2.326),
    (129, 1024, 512, 128, 16, -2.326),
    (500, 520, 2048, 256, 8, -1.645),   # one slice over several lanes' vectors
    (100, 2304, 512, 64, 4, -1.645),    # slices of 288 columns across scale blocks
    (60, 8192, 256, 64, 4, -1.645),
])
def test_backward_matches_oracle(n, dm, dff, T, C, b0, dtype):
    say(f"backward_act8 {dtype} n={n} dm={dm} dff={dff}")
    cfg, t = layer(n, dm, dff, dtype, b0, seed=n + dff)
    dt = cfg.torch_dtype
    x, wu, b, wd = oracle_inputs(t)
    h = torch.from_numpy(oracle.ffn_hidden(x, wu, b)).to(dt)
    x8, codes, scales, _ = on_gpu_pack(t["x"])
    hy, status, g = run_backward(t, x8, h, T, C)
    assert status == twell.TWELL_OK
    ref = oracle.ffn_backward_from_h(act8_decode(codes, scales, dm), as_f64(h), wu, wd,
                                     as_f64(t["dy"]))
    check(g, ref, dt)


@pytest.mark.gpu
def test_backward_widest_rows():
    """16384 bfloat16 columns: two vectors per lane and slice."""
    say("backward_act8 dm=16384")
    n, dm, dff = 20, 16384, 128
    cfg, t = layer(n, dm, dff, "bf16", -1.0, seed=4)
    x, wu, b, wd = oracle_inputs(t)
    h = torch.from_numpy(oracle.ffn_hidden(x, wu, b)).to(torch.bfloat16)
    x8, codes, scales, _ = on_gpu_pack(t["x"])
    _, _, g = run_backward(t, x8, h, 64, 16)
    check(g, oracle.ffn_backward_from_h(act8_decode(codes, scales, dm), as_f64(h), wu, wd,
                                        as_f64(t["dy"])), torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [40, 257, 700])
def test_backward_integer_valued_exact(n, dtype):
    """Codes in -1..1 with scales 1 and 2, small integer weights: every sum is exact."""
    dm, dff, T, C = 512, 2048, 128, 4
    say(f"backward_act8 integer-valued {dtype} n={n}")
    rng = np.random.default_rng(n)

    def tern(shape, zero):
        a = rng.integers(-1, 2, size=shape).astype(np.float32)
        a[rng.random(shape) < zero] = 0
        return a
    t = {"w_up_t": torch.from_numpy(tern((dff, dm), 0.7)).to(dtype),
         "w_down": torch.from_numpy(tern((dff, dm), 0.8)).to(dtype),
         "dy": torch.from_numpy(tern((n, dm), 0.5)).to(dtype)}
    x8 = twell.Act8.empty(n, dm, dtype, "cuda:0")
    x8.codes.copy_(torch.from_numpy(tern((n, dm), 0.7).astype(np.int8)))
    x8.scales.copy_(torch.from_numpy(rng.integers(1, 3, size=(n, 4)).astype(np.float32)))
    x = act8_decode(x8.codes.cpu().numpy(), x8.scales.cpu().numpy(), dm)
    wu, wd, dy = (as_f64(t[k]) for k in ("w_up_t", "w_down", "dy"))
    h = np.maximum(x @ wu.T - 14, 0)
    assert h.max() <= 256
    ht = torch.from_numpy(h).to(dtype)
    hy, status, g = run_backward(t, x8, ht, T, C)
    assert status == twell.TWELL_OK and hy.n_dense_host() > 0
    ref = oracle.ffn_backward_from_h(x, h, wu, wd, dy)
    assert np.abs(np.where(h != 0, dy @ wd.T, 0)).max() <= 256
    np.testing.assert_array_equal(as_f64(g.dw_down), ref.dw_down)
    np.testing.assert_array_equal(as_f64(g.dw_up_t), ref.dw_up_t)
    np.testing.assert_array_equal(as_f64(g.db_up), ref.db)
    np.testing.assert_array_equal(as_f32(g.dx), as_f32(torch.from_numpy(ref.dx).to(dtype)))


@pytest.mark.gpu
def test_backward_against_differences():
    """The directional derivative of L = sum(y * dy) along random weight directions, by central
    differences of the float64 forward at the checkpoint's x, away from the ReLU's kink (steps
    that flip a unit are excluded by their size: the smallest active z is far above the step)."""
    say("backward_act8 differences")
    n, dm, dff = 24, 256, 512
    cfg, t = layer(n, dm, dff, "fp32", -1.0, seed=2)
    x8, codes, scales, _ = on_gpu_pack(t["x"])
    x = act8_decode(codes, scales, dm)
    _, wu, b, wd = oracle_inputs(t)
    dy = as_f64(t["dy"])
    h = np.maximum(x @ wu.T + b, 0)
    h32 = torch.from_numpy(h).float()
    _, _, g = run_backward(t, x8, h32, 64, 8)
    rng = np.random.default_rng(0)
    eps = 1e-7
    loss = lambda u, bb, dn: float((np.maximum(x @ u.T + bb, 0) @ dn * dy).sum())
    for _ in range(3):
        vu, vb, vd = (rng.standard_normal(a.shape) for a in (wu, b, wd))
        fd = (loss(wu + eps * vu, b + eps * vb, wd + eps * vd) -
              loss(wu - eps * vu, b - eps * vb, wd - eps * vd)) / (2 * eps)
        parts = [(as_f64(g.dw_up_t) * vu).sum(), (as_f64(g.db_up) * vb).sum(),
                 (as_f64(g.dw_down) * vd).sum()]
        # a direction's sum is a random walk: compare against the gradient's norm
        norm = np.sqrt(sum((as_f64(a) ** 2).sum() for a in (g.dw_up_t, g.db_up, g.dw_down)))
        assert abs(fd - sum(parts)) <= 1e-3 * norm, (fd, parts)


@pytest.mark.gpu
def test_backward_edges():
    """No rows, no active unit, a dense capacity short of the dense rows, a NaN block."""
    say("backward_act8 edges")
    dm, dff, T, C = 256, 1024, 64, 4
    cfg, t = layer(300, dm, dff, "bf16", -2.326, seed=11)
    x8, codes, scales, _ = on_gpu_pack(t["x"])
    x, wu, b, wd = oracle_inputs(t)
    h = torch.from_numpy(oracle.ffn_hidden(x, wu, b)).to(torch.bfloat16)
    _, _, g = run_backward(t, x8, torch.zeros_like(h), T, C)
    for a in (g.dx, g.dw_up_t, g.db_up, g.dw_down):
        assert not a.float().any()
    e8 = twell.Act8.empty(0, dm, torch.bfloat16, "cuda:0")
    t0 = {k: (v[:0] if k in ("x", "dy") else v) for k, v in t.items()}
    _, _, g = run_backward(t0, e8, h[:0], T, C)
    for a in (g.dw_up_t, g.db_up, g.dw_down):
        assert torch.equal(a, torch.zeros_like(a))
    hy, status, g = run_backward(t, x8, h, T, C, dense_capacity=3)
    assert status == twell.TWELL_ERR_DENSE_CAPACITY
    hs = as_f64(h)
    hs[oracle.pack(as_f32(h), T, C).dense_rows[3:]] = 0
    ref = oracle.ffn_backward_from_h(act8_decode(codes, scales, dm), hs, wu, wd, as_f64(t["dy"]))
    check(g, ref, torch.bfloat16)
    # one row's first block is NaN: it reaches the neurons active in that row, its columns only
    row = int((as_f64(h) != 0).sum(axis=1).argmax())
    x8.scales[row, 0] = float("nan")
    _, _, g = run_backward(t, x8, h, T, C)
    active = as_f64(h)[row] != 0
    nan = torch.isnan(g.dw_up_t).cpu().numpy()
    assert active.any() and nan[active][:, :128].all()
    assert not nan[~active].any() and not nan[:, 128:].any()


@pytest.mark.gpu
def test_backward_repeats_bit_for_bit():
    say("backward_act8 determinism and graph")
    n, dm, dff, T, C = 1000, 512, 2048, 128, 4
    cfg, t = layer(n, dm, dff, "bf16", -1.645, seed=5)
    x, wu, b, _ = oracle_inputs(t)
    h = torch.from_numpy(oracle.ffn_hidden(x, wu, b)).to(torch.bfloat16).cuda()
    d = {k: v.cuda() for k, v in t.items()}
    hy, _ = twell.twell_pack(h, T, C)
    x8 = twell.twell_act8_pack(d["x"])
    ws = twell.backward_act8_workspace(hy, dm)
    run = lambda out: twell.ffn_sparse_backward_act8(x8, d["w_up_t"], d["w_down"], hy, d["dy"],
                                                     out=out, workspace=ws)
    ref = run(None)
    out = run(None)
    fields = lambda g: (g.dx, g.dw_up_t, g.db_up, g.dw_down)
    torch.cuda.synchronize()
    for u, v in zip(fields(ref), fields(out)):
        assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for _ in range(3):
        for a in fields(out):
            a.fill_(7)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(fields(ref), fields(out)):
            assert torch.equal(u, v)


@pytest.mark.gpu
def test_backward_refusals():
    n, dm, dff = 16, 128, 512
    cfg, t = layer(n, dm, dff, "bf16", -1.645, seed=1)
    d = {k: v.cuda() for k, v in t.items()}
    hy, _ = twell.twell_pack(torch.zeros((n, dff), dtype=torch.bfloat16, device="cuda"), 64, 4)
    x8 = twell.twell_act8_pack(d["x"])
    call = lambda a, **kw: twell.ffn_sparse_backward_act8(a, d["w_up_t"], d["w_down"], hy, d["dy"],
                                                          **kw)
    with pytest.raises(ValueError, match="x8 holds"):
        call(twell.twell_act8_pack(d["x"][:8].contiguous()))
    with pytest.raises(ValueError, match="x8 holds"):
        call(twell.twell_act8_pack(d["x"].float()))
    with pytest.raises(twell.TwellError) as e:
        call(x8, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == twell.TWELL_ERR_WORKSPACE
    with pytest.raises(ValueError, match="workspace"):
        call(x8, workspace=torch.empty(1 << 24, dtype=torch.uint8))
