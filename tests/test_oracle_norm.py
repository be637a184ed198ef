"""The oracle of the norms around the layer: hand-worked rows, PyTorch's float64 autograd on the
CPU, and central differences."""
import numpy as np
import pytest
import torch

from oracle.train_oracle import norm, norm_grad


def test_hand_worked():
    r = np.array([[3.0, 4.0]])
    _, x = norm(r, None, None, None, np.array([1.0, 2.0]), 1.0, 0.5)
    np.testing.assert_allclose(x, [[3 / np.sqrt(13), 8 / np.sqrt(13)]])  # mean square 12.5
    out, x = norm(r, np.array([[1.0, -1.0]]), np.array([2.0, 1.0]), np.array([0.5, 3.0]), None,
                  2.0, 3.0)  # y / 2
    np.testing.assert_allclose(out, [[6 + 0.5, 8 - 1.5]])
    assert x is None
    out, _ = norm(r, np.array([[1.0, -1.0]]), None, None, None, 2.0, 3.0)
    np.testing.assert_allclose(out, [[7.0, 7.0]])


@pytest.mark.parametrize("with_y,post,gate,pre,dr", [
    (1, 1, 1, 1, 1), (1, 1, 0, 1, 0), (1, 0, 1, 1, 1), (1, 0, 0, 0, 1), (1, 1, 1, 0, 1),
    (0, 0, 0, 1, 1), (0, 0, 0, 1, 0)])
def test_gradients(with_y, post, gate, pre, dr):
    rng = np.random.default_rng(5)
    n, d, alpha, eps = 6, 10, (0.7 if with_y else 1.0), 0.01
    given = {"residual": rng.normal(size=(n, d)), "y": rng.normal(size=(n, d)) if with_y else None,
             "w_post": rng.normal(size=d) if post else None,
             "gate": rng.normal(size=d) if gate else None,
             "w_pre": rng.normal(size=d) if pre else None}
    upr = rng.normal(size=(n, d)) if dr else None
    upx = rng.normal(size=(n, d)) if pre else None

    def loss(p):
        r, x = norm(p["residual"], p["y"], p["w_post"], p["gate"], p["w_pre"], alpha, eps)
        return (0 if upr is None else (r * upr).sum()) + (0 if upx is None else (x * upx).sum())

    rout, _ = norm(given["residual"], given["y"], given["w_post"], given["gate"], given["w_pre"],
                   alpha, eps)
    got = norm_grad(rout, given["y"], given["w_post"], given["gate"], given["w_pre"], upr, upx,
                    alpha, eps)
    names = dict(residual="d_residual", y="dy", w_post="dw_post", gate="dgate", w_pre="dw_pre")
    leaves = {k: torch.tensor(v, requires_grad=True) for k, v in given.items() if v is not None}
    r = leaves["residual"]
    if with_y:
        u = leaves["y"]
        if post:
            u = u * torch.rsqrt(u.square().mean(1, keepdim=True) + eps) * leaves["w_post"]
        r = alpha * r + (u * leaves["gate"] if gate else u)
    total = 0 if upr is None else (r * torch.tensor(upr)).sum()
    if pre:
        x = r * torch.rsqrt(r.square().mean(1, keepdim=True) + eps) * leaves["w_pre"]
        total = total + (x * torch.tensor(upx)).sum()
    auto = dict(zip(leaves, torch.autograd.grad(total, list(leaves.values()))))
    for k, name in names.items():
        if given[k] is None:
            assert name not in got
            continue
        np.testing.assert_allclose(got[name], auto[k].numpy(), rtol=1e-10, atol=1e-12)
        assert np.all(got["of_" + name] >= np.abs(got[name]) - 1e-12)
        flat = given[k].reshape(-1)
        for i in range(0, flat.size, 7):
            h, keep = 1e-6, flat[i]
            flat[i] = keep + h
            up = loss(given)
            flat[i] = keep - h
            down = loss(given)
            flat[i] = keep
            assert abs((up - down) / (2 * h) - got[name].reshape(-1)[i]) < 1e-7
