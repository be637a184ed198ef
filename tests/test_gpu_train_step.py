"""The training-step example end to end, and its gradients against PyTorch's autograd in float64
on the same weights (8-bit input and bfloat16 storage apart)."""
import importlib.util
import math
import os

import pytest
import torch

from activation_sparse_transformer_amd import twell
from gpu_helpers import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("train_step",
                                                  os.path.join(ROOT, "examples", "train_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_loss_falls(example):
    """From log(vocab) towards the noise's own entropy (0.1 log 1000 + h(0.1), about 1.0)."""
    losses = example.train(60, 4096, say=say)
    assert abs(losses[0] - math.log(example.VOCAB)) < 1.5
    assert losses[-1] < 2.5 and losses[-1] < 0.5 * losses[0]


def test_step_gradients_match_autograd(example):
    """The whole chain's gradients, against float64 autograd of the same function.  The chain
    stores x, h, y, the logits' gradient and dout in bfloat16 and x in 8 bits (an error of about
    0.006 of x's size), so whole gradients are compared by their 2-norm within 3%."""
    g = torch.Generator().manual_seed(3)
    m = example.Model(g)
    text = example.synthetic_text(512, g)
    tokens, targets = text[:-1].cuda(), text[1:].cuda()
    got = {}
    m.update = lambda grads, lr, t: got.update(grads)
    m.step(tokens, targets, 0.0, 1)
    torch.cuda.synchronize()
    p = {k: v.double().cpu().requires_grad_(True) for k, v in m.p.items()}
    x = p["embed"][tokens.cpu()] * m.scale
    y = torch.relu(x @ p["w_up_t"].t() + p["b_up"]) @ p["w_down"]
    logits = (x + y) @ p["embed"].t() * example.LOGIT_SCALE
    logp = torch.log_softmax(logits, 1).gather(1, targets.cpu()[:, None]).mean()
    grads = torch.autograd.grad(-logp, list(p.values()))
    for (k, ref) in zip(p, grads):
        off = float((got[k].double().cpu() - ref).norm() / ref.norm())
        say(f"{k}: {off:.4f}")
        assert off < 0.03, (k, off)


def test_single_token(example):
    say("one token through the whole chain")
    m = example.Model(torch.Generator().manual_seed(1))
    loss = m.step(torch.tensor([5], device="cuda"), torch.tensor([38], device="cuda"), 0.01, 1)
    assert math.isfinite(loss)
    out = list(m.continue_prompt(5, 2))
    assert len(out) == 2 and all(0 <= t < example.VOCAB for t, _, _ in out)
