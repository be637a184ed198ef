"""GPU parity of the token embedding (twell_embed_forward) and its gradient
(twell_embed_backward) against the CPU oracle.

Lookup: one float32 product rounded once, equal bit for bit to that computed on the host.
Gradient: float32 sums of k terms in some fixed order are within k * 2^-24 of the sum of
magnitudes, and the scale's product adds one rounding; the integer-valued cases are exact."""
import ctypes

import numpy as np
import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import as_f32, as_f64, say, u32
from oracle.train_oracle import embed, embed_grad

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])


def token_ids(seed, n, vocab, index, kind):
    """Ids with repeats and (all kinds but `same`) some outside the table."""
    rng = np.random.default_rng(seed)
    if kind == "zipf":
        t = np.exp(rng.random(n) * np.log(vocab + 1)).astype(np.int64) - 1
    elif kind == "same":
        return torch.full((n,), vocab - 1, dtype=index)
    elif kind == "none":
        t = np.full(n, -1, np.int64)
    else:  # every id once, in some order, then repeats
        t = np.concatenate([rng.permutation(vocab)] * (n // vocab + 1))[:n]
    t = np.minimum(t, vocab - 1)
    bad = rng.random(n) < 0.05
    t[bad] = rng.choice([-1, -100, vocab, vocab + 5], bad.sum())
    return torch.from_numpy(t).to(index)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,vocab,d,scale,index", [
    (1, 1, 8, 1.0, torch.int64), (3, 7, 24, 45.25, torch.int32), (16, 5000, 4096, 1.0, torch.int64),
    (1000, 333, 520, 0.3, torch.int32), (77, 100, 8200, 90.5, torch.int64)])
def test_lookup_exact(n, vocab, d, scale, index, dtype):
    say(f"embed {dtype} n={n} vocab={vocab} d={d}")
    g = torch.Generator().manual_seed(n)
    table = torch.randn((vocab, d), generator=g).to(dtype)
    t = token_ids(n, n, vocab, index, "zipf")
    got = twell.twell_embed_forward(table.cuda(), t.cuda(), scale=scale)
    torch.cuda.synchronize()
    ok = (t >= 0) & (t < vocab)
    rows = table[t.long().clamp(0, vocab - 1)].float() * np.float32(scale)
    want = torch.where(ok[:, None], rows, torch.zeros(())).to(dtype)
    np.testing.assert_array_equal(u32(as_f32(got)), u32(as_f32(want)))
    ref = embed(as_f64(table), t.numpy(), scale)
    eps = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
    assert np.all(np.abs(as_f64(got) - ref) <= eps * np.abs(ref))


def run_grad(dout, t, vocab, scale):
    out = torch.full((vocab, dout.shape[1]), float("nan"), device="cuda")
    got = twell.twell_embed_backward(dout.cuda(), t.cuda(), vocab, scale=scale, out=out)
    torch.cuda.synchronize()
    return as_f64(got)


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,vocab,d,kind,index", [
    (1, 1, 8, "zipf", torch.int64),
    (64, 3, 128, "zipf", torch.int32),       # segments of about a wave's length
    (65, 1, 136, "same", torch.int64),       # the shortest long segment
    (64, 1, 136, "same", torch.int64),       # the longest short one
    (500, 40, 520, "zipf", torch.int64),
    (3000, 7, 264, "each", torch.int32),
    (5000, 20000, 256, "zipf", torch.int64),
    (4097, 4097, 64, "each", torch.int64),
    (40000, 1000, 64, "zipf", torch.int32),  # several windows of token numbers
    (40000, 5, 8, "same", torch.int64),
    (200, 9000, 1032, "none", torch.int64),
    (8192, 100000, 64, "zipf", torch.int32),   # the most tokens and ids that one workgroup sorts
    (8193, 100000, 64, "zipf", torch.int64),
    (700, (1 << 19) - 1, 8, "zipf", torch.int64),
    (700, 1 << 19, 8, "zipf", torch.int64),
    (600000, 700000, 8, "zipf", torch.int32),  # past one bitmap of token numbers
    (513, 600, 16, "same", torch.int64)])
def test_gradient_matches_oracle(n, vocab, d, kind, index, dtype):
    say(f"embed grad {dtype} n={n} vocab={vocab} d={d} {kind}")
    g = torch.Generator().manual_seed(n + d)
    dout = torch.randn((n, d), generator=g).to(dtype)
    t = token_ids(n + vocab, n, vocab, index, kind)
    got = run_grad(dout, t, vocab, 1.7)
    ids = t.numpy()
    ref = embed_grad(as_f64(dout), ids, vocab, np.float64(np.float32(1.7)))
    size = embed_grad(np.abs(as_f64(dout)), ids, vocab, 1.7)
    k = np.bincount(ids[(ids >= 0) & (ids < vocab)], minlength=vocab)[:, None]
    assert np.all(np.abs(got - ref) <= (k + 1) * 2.0 ** -24 * size)
    assert not got[k[:, 0] == 0].any()


@pytest.mark.gpu
@BOTH
@pytest.mark.parametrize("n,vocab,kind", [(3000, 50, "zipf"), (20000, 3, "same"),
                                          (700, 2000, "each")])
def test_gradient_integer_valued_exact(n, vocab, kind, dtype):
    say(f"embed grad exact {dtype} n={n} {kind}")
    d = 72
    rng = np.random.default_rng(n)
    dout = torch.from_numpy(rng.integers(-3, 4, (n, d)).astype(np.float32)).to(dtype)
    t = token_ids(5, n, vocab, torch.int64, kind)
    np.testing.assert_array_equal(run_grad(dout, t, vocab, 0.5),
                                  embed_grad(as_f64(dout), t.numpy(), vocab, 0.5))


@pytest.mark.gpu
def test_gradient_against_differences():
    """L = sum(out * w) is linear in the table: its difference along a direction is exact up to
    the float64 rounding of the two values."""
    say("embed grad differences")
    n, vocab, d, scale = 300, 50, 64, 2.0
    g = torch.Generator().manual_seed(1)
    w = torch.randn((n, d), generator=g)
    t = token_ids(1, n, vocab, torch.int64, "zipf")
    got = run_grad(w, t, vocab, scale)
    rng = np.random.default_rng(2)
    table, v = rng.standard_normal((2, vocab, d))
    loss = lambda tab: (embed(tab, t.numpy(), scale) * as_f64(w)).sum()
    fd = (loss(table + v) - loss(table - v)) / 2
    assert abs(fd - (got * v).sum()) <= 1e-5 * np.abs(got * v).sum()


@pytest.mark.gpu
@pytest.mark.parametrize("index", [torch.int32, torch.int64])
def test_part_of_a_longer_text(index):
    """Ids that start anywhere in their own array."""
    say(f"embed unaligned ids {index}")
    text = token_ids(4, 300, 40, index, "zipf").cuda()
    table = torch.randn((40, 64), device="cuda")
    for first in (1, 2, 3):
        part = text[first:]
        assert torch.equal(twell.twell_embed_forward(table, part),
                           twell.twell_embed_forward(table, part.clone()))
        dout = torch.randn((len(part), 64), device="cuda")
        assert torch.equal(twell.twell_embed_backward(dout, part, 40),
                           twell.twell_embed_backward(dout, part.clone(), 40))


@pytest.mark.gpu
def test_special_values_stay_in_their_rows():
    """NaN and infinite gradients reach their own id only; no token leaves the table zero."""
    say("embed special values")
    n, vocab, d = 200, 30, 64
    t = token_ids(3, n, vocab, torch.int64, "zipf")
    dout = torch.ones((n, d))
    i = int(torch.nonzero((t >= 0) & (t < vocab))[0])
    dout[i, 5] = float("nan")
    got = run_grad(dout, t, vocab, 1.0)
    nan = np.zeros((vocab, d), bool)
    nan[int(t[i]), 5] = True
    np.testing.assert_array_equal(np.isnan(got), nan)
    empty = run_grad(torch.empty((0, d)), torch.empty((0,), dtype=torch.int64), vocab, 1.0)
    np.testing.assert_array_equal(empty, np.zeros((vocab, d)))
    out = twell.twell_embed_forward(torch.ones((4, 8), device="cuda"),
                                    torch.empty((0,), dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 8)


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """A table of more than 2^31 elements: its last rows are read and written."""
    say("embed offsets past 2^31")
    d, vocab = 8192, 270000
    t = torch.tensor([vocab - 1, 0, vocab - 2, vocab - 1], device="cuda")
    table = torch.empty((vocab, d), dtype=torch.bfloat16, device="cuda")
    table[0], table[vocab - 2], table[vocab - 1] = 1.0, 2.0, 3.0
    out = twell.twell_embed_forward(table, t)
    assert out.float().mean(1).tolist() == [3.0, 1.0, 2.0, 3.0]
    del table
    grad = twell.twell_embed_backward(out, t, vocab)
    torch.cuda.synchronize()
    assert torch.equal(grad[vocab - 1], torch.full((d,), 6.0, device="cuda"))
    assert torch.equal(grad[vocab - 2], torch.full((d,), 2.0, device="cuda"))
    assert torch.equal(grad[0], torch.full((d,), 1.0, device="cuda"))
    assert int(torch.count_nonzero(grad[1:vocab - 2])) == 0


@pytest.mark.gpu
def test_repeats_bit_for_bit_and_in_graphs():
    say("embed determinism, graph, side stream")
    n, vocab, d = 20000, 3000, 128
    g = torch.Generator().manual_seed(7)
    dout = torch.randn((n, d), generator=g).cuda()
    t = token_ids(8, n, vocab, torch.int64, "zipf").cuda()
    table = torch.randn((vocab, d), generator=g).to(torch.bfloat16).cuda()
    ws = twell.embed_backward_workspace(n, d, vocab, "cuda")
    ref = twell.twell_embed_backward(dout, t, vocab)
    fwd = twell.twell_embed_forward(table, t)
    out, fout = torch.empty_like(ref), torch.empty_like(fwd)

    def both():
        twell.twell_embed_backward(dout, t, vocab, out=out, workspace=ws)
        twell.twell_embed_forward(table, t, out=fout)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        both()
    side.synchronize()
    assert torch.equal(out, ref) and torch.equal(fout, fwd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(3):
        out.fill_(7)
        fout.fill_(7)
        ws.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(fout, fwd)


@pytest.mark.gpu
def test_refusals():
    table = torch.zeros((10, 64), dtype=torch.bfloat16, device="cuda")
    t = torch.zeros((4,), dtype=torch.int64, device="cuda")
    dout = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="int32 or int64"):
        twell.twell_embed_forward(table, t.short())
    with pytest.raises(ValueError, match="not supported"):
        twell.twell_embed_forward(table.half(), t)
    with pytest.raises(ValueError, match="contiguous"):
        twell.twell_embed_forward(table[:, :32], t)
    with pytest.raises(ValueError, match="tokens must have shape"):
        twell.twell_embed_backward(dout, t[:3], 10)
    with pytest.raises(ValueError, match="out must be"):
        twell.twell_embed_backward(dout, t, 10, out=torch.zeros_like(table))
    for bad in (lambda: twell.twell_embed_forward(table, t, scale=float("nan")),
                lambda: twell.twell_embed_backward(dout, t, 0),
                lambda: twell.twell_embed_forward(table[:, :60].contiguous(), t)):
        with pytest.raises(twell.TwellError) as e:
            bad()
        assert e.value.code == twell.TWELL_ERR_INVALID_ARG
    with pytest.raises(twell.TwellError) as e:
        twell.twell_embed_backward(dout, t, 10,
                                   workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.code == twell.TWELL_ERR_WORKSPACE


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="fake device pointers are passed only on a GPU-less host")
def test_host_checks():
    lib = twell.load()
    p = 4096
    bad = twell.TWELL_ERR_INVALID_ARG

    def shape(**kw):
        f = dict(n_tokens=4, vocab=10, d_model=64, dtype=1, index_bytes=8, scale=1.0, reserved=0)
        return twell.EmbedShape(**{**f, **kw})
    fwd = lambda s, *a: lib.twell_embed_forward(ctypes.byref(s), *a, None)
    for kw in (dict(n_tokens=-1), dict(n_tokens=1 << 31), dict(vocab=0), dict(d_model=12),
               dict(dtype=3), dict(index_bytes=2), dict(scale=float("inf")), dict(reserved=1)):
        assert fwd(shape(**kw), p, p, p) == bad, kw
        assert lib.twell_embed_backward_workspace_size(ctypes.byref(shape(**kw))) == 0
    assert fwd(shape(), None, p, p) == bad and fwd(shape(), p, p + 4, p) == bad and fwd(shape(), p + 8, p, p) == bad
    assert lib.twell_embed_forward(None, p, p, p, None) == bad
    need = lib.twell_embed_backward_workspace_size(ctypes.byref(shape()))
    bwd = lambda *a: lib.twell_embed_backward(ctypes.byref(shape()), *a, None)
    assert bwd(p, p, p, p, need - 1) == twell.TWELL_ERR_WORKSPACE
    assert bwd(p, p, p, None, need) == bad and bwd(p, p, None, p, need) == bad
    assert bwd(p, p, p + 4, p, need) == bad
    assert fwd(shape(n_tokens=0), None, None, None) == twell.TWELL_OK
