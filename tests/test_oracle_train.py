"""The training-step oracle against hand-worked values and PyTorch's float64 autograd (CPU)."""
import numpy as np
import torch

from oracle.train_oracle import (act8_decode, act8_quotients, embed, embed_grad, logprob,
                                 logprob_grad)


def test_act8_by_hand():
    x = np.zeros((2, 130))
    x[0, :3] = [2.0, -1.0, 0.5]      # a = 2: quotients 127, -63.5, 31.75
    x[0, 128] = -4.0                 # the short last block has its own scale
    q, a = act8_quotients(x)
    assert a.tolist() == [[2.0, 4.0], [0.0, 0.0]]
    assert q[0, :3].tolist() == [127.0, -63.5, 31.75] and q[0, 128] == -127.0 and not q[1].any()
    codes, scales = np.rint(q).astype(np.int8), a / 127
    assert codes[0, :3].tolist() == [127, -64, 32]  # ties to even
    back = act8_decode(codes, scales, 130)
    assert np.abs(back - x).max() <= 2.0 / 254 + 1e-12


def test_embed_by_hand():
    table = np.arange(6.0).reshape(3, 2)
    t = np.array([2, -1, 0, 2, 3])
    np.testing.assert_array_equal(embed(table, t, 2.0),
                                  [[8, 10], [0, 0], [0, 2], [8, 10], [0, 0]])
    d = np.ones((5, 2)) * np.arange(1, 6)[:, None]
    np.testing.assert_array_equal(embed_grad(d, t, 3, 0.5), [[1.5, 1.5], [0, 0], [2.5, 2.5]])


def test_logprob_by_hand():
    """Two equal places and a masked one: probabilities one half, entropy log 2."""
    x = np.array([[3.0, -np.inf, 3.0], [-np.inf] * 3, [0.0, 0.0, np.log(2.0)]])
    logp, entropy, lse, ids, tops = logprob(x, np.array([2, 0, -1]), 1.0, 2)
    np.testing.assert_allclose(logp, [-np.log(2), -np.inf, 0.0])
    np.testing.assert_allclose(entropy, [np.log(2), 0.0, 1.5 * np.log(2)])
    np.testing.assert_allclose(lse, [3 + np.log(2), -np.inf, np.log(4)])
    assert ids.tolist() == [[0, 2], [-1, -1], [2, 0]]
    np.testing.assert_allclose(tops, [[-np.log(2)] * 2, [-np.inf] * 2, [-np.log(2), -np.log(4)]])


def test_logprob_and_gradient_against_autograd():
    rng = np.random.default_rng(0)
    n, v, scale = 7, 40, 1.3
    x = rng.standard_normal((n, v)) * 3
    t = rng.integers(0, v, n)
    t[2] = -1
    g, w = rng.standard_normal((2, n))
    z = torch.tensor(x, requires_grad=True)
    lp = torch.log_softmax(z * scale, 1)
    at = lp.gather(1, torch.tensor(np.maximum(t, 0))[:, None])[:, 0] * torch.tensor(t >= 0)
    ent = -(lp.exp() * lp).sum(1)
    ref = torch.autograd.grad((at * torch.tensor(g) + ent * torch.tensor(w)).sum(), z)[0]
    logp, entropy, lse, _, _ = logprob(x, t, scale, 0)
    np.testing.assert_allclose(logp, at.detach(), atol=1e-12)
    np.testing.assert_allclose(entropy, ent.detach(), atol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(z * scale, 1).detach(), atol=1e-12)
    np.testing.assert_allclose(logprob_grad(x, t, scale, g, w), ref, atol=1e-12)
