"""The output head on the kernels that large calls take: 256 x 256 tiles over several stages of K,
with remainders in every dimension.  Bounds: test_gpu_head's."""
import pytest
import torch

from gpu_helpers import say
from test_gpu_head import BOTH, check, make

pytestmark = pytest.mark.gpu
# n, vocab, d: every product of the first takes 256 x 256 tiles in both types, the others mix them
# (test_cut_rules.py)
LARGE = [(1891, 5395, 1448)]
MIXED = [(2500, 5000, 456), (1175, 6917, 1000), (520, 9001, 712)]


@BOTH
@pytest.mark.parametrize("n,v,d", LARGE + MIXED)
def test_large_tiles(n, v, d, dtype):
    say(f"head tiles {dtype} n={n} v={v} d={d}")
    check(make(n + v + d, n, v, d, dtype, 0.7))


@BOTH
def test_repeats(dtype):
    """The same bits again, whatever the workspaces held."""
    from activation_sparse_transformer_amd import twell
    n, v, d = LARGE[0]
    m = make(3, n, v, d, dtype)
    x, w, t, c = m["x"].cuda(), m["w"].cuda(), m["t"].cuda(), m["dlogp"].cuda()
    ws = [twell.head_logprob_workspace(n, v, d, dtype, "cuda", backward=b) for b in (False, True)]

    def run():
        f = twell.twell_head_logprob_forward(x, w, t, workspace=ws[0])
        g = twell.twell_head_logprob_backward(x, w, t, f.stats, c, workspace=ws[1])
        return [*vars(f).values(), *vars(g).values()]
    first = run()
    for fill in (0, 255, 63):
        for s in ws:
            s.fill_(fill)
        assert all(torch.equal(a, b) for a, b in zip(first, run()))


@BOTH
@pytest.mark.parametrize("n,v", [(1, 1500), (5, 9000), (16, 1500), (30, 9000), (64, 1500)])
def test_few_rows_replayed(n, v, dtype):
    """The kernels of few rows, captured and replayed on other values."""
    from activation_sparse_transformer_amd import twell
    say(f"head replayed {dtype} n={n} v={v}")
    d = 72
    m = make(5, n, v, d, dtype)
    x, w, t, c = m["x"].cuda(), m["w"].cuda(), m["t"].cuda(), m["dlogp"].cuda()
    ws = [twell.head_logprob_workspace(n, v, d, dtype, "cuda", backward=b) for b in (False, True)]

    def run():
        f = twell.twell_head_logprob_forward(x, w, t, workspace=ws[0])
        g = twell.twell_head_logprob_backward(x, w, t, f.stats, c, workspace=ws[1])
        return [*vars(f).values(), *vars(g).values()]
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for seed in (6, 7, 8):
        o = make(seed, n, v, d, dtype)
        x.copy_(o["x"]), w.copy_(o["w"]), t.copy_(o["t"]), c.copy_(o["dlogp"])
        ref = [a.clone() for a in run()]
        for s in ws:
            s.fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    del graph


@BOTH
def test_two_calls_at_once(dtype):
    """Two streams, each with workspaces of its own, side by side."""
    from activation_sparse_transformer_amd import twell
    sizes = [(300, 4000, 520), (16, 4000, 520)]
    given = []
    for i, (n, v, d) in enumerate(sizes):
        m = make(i, n, v, d, dtype)
        given.append([m[k].cuda() for k in ("x", "w", "t", "dlogp")])

    def run(x, w, t, c):
        f = twell.twell_head_logprob_forward(x, w, t)
        return [*vars(f).values(), *vars(twell.twell_head_logprob_backward(x, w, t, f.stats,
                                                                           c)).values()]
    ref = [run(*g) for g in given]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sizes]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(*given[i]))
    torch.cuda.synchronize()
    for r, all_of in zip(ref, got):
        for g in all_of:
            assert all(torch.equal(a, b) for a, b in zip(r, g))
