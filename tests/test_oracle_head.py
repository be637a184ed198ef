"""The oracle of the output head's log probabilities: hand-worked rows and PyTorch's float64
autograd on the CPU."""
import numpy as np
import torch

from oracle.train_oracle import head_logprob, head_logprob_grad


def test_hand_worked():
    x = np.array([[1.0, 2.0], [0.0, 1.0]])
    w = np.array([[1.0, 0.0], [0.0, 1.0], [1.0, 1.0]])
    logp, lse, stats, z = head_logprob(x, w, np.array([1, -1]), 2.0)
    np.testing.assert_allclose(z, [[2, 4, 6], [0, 2, 2]])
    np.testing.assert_allclose(stats[0], [6, 1 + np.exp(-2) + np.exp(-4)])
    np.testing.assert_allclose(logp, [4 - lse[0], 0])
    np.testing.assert_allclose(lse[1], np.log(1 + 2 * np.exp(2)))


def test_gradient_is_autograds():
    g = torch.Generator().manual_seed(2)
    x = torch.randn((7, 5), generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn((11, 5), generator=g, dtype=torch.float64, requires_grad=True)
    t = torch.tensor([0, 10, -100, 3, 3, 11, 5])
    c = torch.randn(7, generator=g, dtype=torch.float64)
    ok = (t >= 0) & (t < 11)
    lp = torch.log_softmax(0.7 * x @ w.t(), 1)
    loss = (lp[torch.arange(7), t.clamp(0, 10)] * c * ok).sum()
    dx, dw = torch.autograd.grad(loss, [x, w])
    c[~ok] = float("nan")
    got = head_logprob_grad(x.detach().numpy(), w.detach().numpy(), t.numpy(), c.numpy(), 0.7)
    np.testing.assert_allclose(got[0], dx.numpy(), atol=1e-14)
    np.testing.assert_allclose(got[1], dw.numpy(), atol=1e-14)
