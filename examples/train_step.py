"""Train a one-layer ReLU-sparse language model on synthetic text with the library's operators.

    python examples/train_step.py [--steps 60] [--tokens 4096] [--block]

One step runs them as a training loop does: the embedding (twell_embed_forward), the layer with
its hidden activations in hybrid TwELL form (ffn_sparse_forward), its input kept as an 8-bit
checkpoint (twell_act8_pack), the log probabilities of the next tokens and their gradient
(twell_logprob_forward, twell_logprob_backward), the layer's backward from the checkpoint
(ffn_sparse_backward_act8) and the embedding's gradient (twell_embed_backward).  PyTorch holds
the tensors, multiplies the output head and updates the weights.  Afterwards the model continues
a prompt token by token and prints each token's log probability beside its alternatives.

With --block the layer stands between norms with a gate (twell_norm_forward,
twell_norm_backward), the loss and its gradient come from the hidden states without logits
(twell_head_logprob_forward, twell_head_logprob_backward), and the layer's matrices take
orthogonalised updates of their momentum (twell_orthogonalize).

The text is a cycle of tokens with noise, so the loss falls from log(vocab) to the noise's own.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from activation_sparse_transformer_amd import twell  # noqa: E402

VOCAB, D_MODEL, D_FF, TILE, CAPACITY, NOISE = 1000, 256, 1024, 64, 16, 0.1
LOGIT_SCALE = 0.25  # the tied head starts with each token's own logit far ahead


def synthetic_text(n: int, g: torch.Generator) -> torch.Tensor:
    """n + 1 tokens of the cycle t -> (7 t + 3) mod VOCAB, each step random with chance NOISE."""
    jump = torch.rand(n + 1, generator=g) < NOISE
    t, out = int(torch.randint(VOCAB, (1,), generator=g)), []
    rand = torch.randint(VOCAB, (n + 1,), generator=g)
    for i in range(n + 1):
        t = int(rand[i]) if jump[i] else (7 * t + 3) % VOCAB
        out.append(t)
    return torch.tensor(out)


class Model:
    """Embedding, one sparse feed-forward layer with a residual, a tied output head; float32
    master weights, bfloat16 compute."""

    def __init__(self, g: torch.Generator):
        w = lambda *s, std: (torch.randn(s, generator=g) * std).cuda()
        self.master = {"embed": w(VOCAB, D_MODEL, std=D_MODEL ** -0.5),
                       "w_up_t": w(D_FF, D_MODEL, std=D_MODEL ** -0.5),
                       "b_up": torch.full((D_FF,), -0.5, device="cuda"),
                       "w_down": w(D_FF, D_MODEL, std=0.1 * D_FF ** -0.5)}
        self.state = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in self.master.items()}
        self.scale = math.sqrt(D_MODEL)
        self.cast()

    def cast(self) -> None:
        self.p = {k: v if k == "b_up" else v.bfloat16() for k, v in self.master.items()}

    def forward(self, tokens: torch.Tensor):
        p = self.p
        x = twell.twell_embed_forward(p["embed"], tokens, scale=self.scale)
        f = twell.ffn_sparse_forward(x, p["w_up_t"], p["b_up"], p["w_down"], TILE, CAPACITY)
        out = x + f.y
        return x, f, out, out @ p["embed"].t()

    def step(self, tokens: torch.Tensor, targets: torch.Tensor, lr: float, t: int) -> float:
        p, n = self.p, tokens.shape[0]
        x, f, out, logits = self.forward(tokens)
        x8 = twell.twell_act8_pack(x)
        del x  # the backward reads the checkpoint
        lp = twell.twell_logprob_forward(logits, targets, scale=LOGIT_SCALE)
        # loss = -mean logp: the gradient with respect to each logp
        dlogp = torch.full((n,), -1.0 / n, device="cuda")
        dlogits = twell.twell_logprob_backward(logits, targets, lp.lse, lp.entropy, dlogp,
                                               scale=LOGIT_SCALE, out=logits)
        dout = dlogits @ p["embed"]
        g = twell.ffn_sparse_backward_act8(x8, p["w_up_t"], p["w_down"], f.hybrid, dout)
        dembed = twell.twell_embed_backward(dout + g.dx, tokens, VOCAB, scale=self.scale)
        dembed += (dlogits.t() @ out).float()  # the tied head's share
        self.update({"embed": dembed, "w_up_t": g.dw_up_t, "b_up": g.db_up,
                     "w_down": g.dw_down}, lr, t)
        return -float(lp.logp.mean())

    def update(self, grads: dict, lr: float, t: int) -> None:
        """Adam."""
        for k, g in grads.items():
            m, v = self.state[k]
            m.mul_(0.9).add_(g, alpha=0.1)
            v.mul_(0.99).addcmul_(g, g, value=0.01)
            self.master[k].sub_(lr * (m / (1 - 0.9 ** t))
                                / ((v / (1 - 0.99 ** t)).sqrt() + 1e-8))
        self.cast()

    def continue_prompt(self, token: int, n: int):
        """n greedy tokens after `token`: (token, log probability, alternatives)."""
        for _ in range(n):
            t = torch.tensor([token], device="cuda")
            logits = self.forward(t)[3]
            lp = twell.twell_logprob_forward(logits, t, top=3, scale=LOGIT_SCALE)
            token = int(lp.top_ids[0, 0])
            yield token, float(lp.top_logp[0, 0]), lp.top_ids[0, 1:].tolist()


class BlockModel(Model):
    """The layer as a block: r = embedding, x = norm(r) w_pre, r' = r + gate norm(ffn(x)) w_post,
    and the head on norm(r') w_final.  The norms' weights are float32."""

    def __init__(self, g: torch.Generator, dtype: torch.dtype = torch.bfloat16):
        self.dtype = dtype
        super().__init__(g)
        for k, v in (("w_pre", 1.0), ("w_post", 1.0), ("gate", 0.5), ("w_final", 1.0)):
            self.master[k] = torch.full((D_MODEL,), v, device="cuda")
            self.state[k] = (torch.zeros_like(self.master[k]), torch.zeros_like(self.master[k]))
        self.cast()

    def cast(self) -> None:
        self.p = {k: v.to(self.dtype) if v.dim() == 2 else v for k, v in self.master.items()}

    def hidden(self, tokens: torch.Tensor):
        p = self.p
        r = twell.twell_embed_forward(p["embed"], tokens, scale=self.scale)
        x = twell.twell_norm_forward(r, w_pre=p["w_pre"]).x
        f = twell.ffn_sparse_forward(x, p["w_up_t"], p["b_up"], p["w_down"], TILE, CAPACITY)
        end = twell.twell_norm_forward(r, f.y, w_post=p["w_post"], gate=p["gate"],
                                       w_pre=p["w_final"])
        return r, x, f, end

    def forward(self, tokens: torch.Tensor):
        r, x, f, end = self.hidden(tokens)
        return x, f, end.x, end.x @ self.p["embed"].t()

    def gradients(self, tokens: torch.Tensor, targets: torch.Tensor):
        """The log probabilities and every weight's gradient of -mean logp."""
        p, n = self.p, tokens.shape[0]
        r, x, f, end = self.hidden(tokens)
        lp = twell.twell_head_logprob_forward(end.x, p["embed"], targets, scale=LOGIT_SCALE)
        dlogp = torch.full((n,), -1.0 / n, device="cuda")
        head = twell.twell_head_logprob_backward(end.x, p["embed"], targets, lp.stats, dlogp,
                                                 scale=LOGIT_SCALE)
        e = twell.twell_norm_backward(end.residual, f.y, None, head.dx, w_post=p["w_post"],
                                      gate=p["gate"], w_pre=p["w_final"])
        g = twell.ffn_sparse_backward(x, p["w_up_t"], p["w_down"], f.hybrid, e.dy)
        s = twell.twell_norm_backward(r, None, e.d_residual, g.dx, w_pre=p["w_pre"])
        dembed = twell.twell_embed_backward(s.d_residual, tokens, VOCAB, scale=self.scale)
        return lp, {"embed": dembed + head.dw, "w_up_t": g.dw_up_t, "b_up": g.db_up,
                    "w_down": g.dw_down, "w_pre": s.dw_pre, "w_post": e.dw_post,
                    "gate": e.dgate, "w_final": e.dw_pre}

    def step(self, tokens: torch.Tensor, targets: torch.Tensor, lr: float, t: int) -> float:
        lp, grads = self.gradients(tokens, targets)
        self.update(grads, lr, t)
        return -float(lp.logp.mean())

    def update(self, grads: dict, lr: float, t: int) -> None:
        """The layer's matrices by orthogonalised momentum, of Adam's size (0.2 an element);
        Adam for the rest."""
        grads = dict(grads)
        for k in ("w_up_t", "w_down"):
            w, m = self.master[k], self.state[k][0]
            m.mul_(0.9).add_(grads.pop(k))
            w.sub_(lr * twell.twell_orthogonalize(m, scale=0.2 * math.sqrt(max(w.shape))))
        super().update(grads, lr, t)


def train(steps: int, tokens: int, seed: int = 0, say=print, model_type=Model) -> list[float]:
    g = torch.Generator().manual_seed(seed)
    model, losses = model_type(g), []
    for t in range(1, steps + 1):
        text = synthetic_text(tokens, g).cuda()
        losses.append(model.step(text[:-1].contiguous(), text[1:].contiguous(), 0.01, t))
        if t == 1 or t % 10 == 0:
            say(f"step {t:4d}  loss {losses[-1]:.3f}  (log vocab {math.log(VOCAB):.3f})")
    token = int(synthetic_text(1, g)[0])
    for nxt, logp, others in model.continue_prompt(token, 5):
        want = (7 * token + 3) % VOCAB
        say(f"{token} -> {nxt} (log p {logp:.2f}, then {others}; the cycle's next is {want})")
        token = nxt
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--block", action="store_true")
    a = ap.parse_args()
    train(a.steps, a.tokens, model_type=BlockModel if a.block else Model)
