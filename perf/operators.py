"""The cases of the training-step operators around the sparse feed-forward layer.

Operators: the embedding lookup with scaling and its gradient, log probabilities of
given tokens (with entropy and top alternatives) and their gradient, 8-bit activation
checkpoints, and the layer's backward pass that reads its input from one.

Where ``own`` is false, ``run`` computes them in elementary torch operations in float32;
where it is true, it calls the library.  ``exact`` computes them in float64.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 128  # columns that share one scale in an 8-bit checkpoint


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the embedding of one decoding step's 16 tokens: latency alone
        dict(name="embed_decode", op="embed", n=16, d=4096, v=32768, dtype="bf16", scale=1.0),
        # a long prefill or a training batch at the widest model, scaled by sqrt(d_model)
        dict(name="embed_batch", op="embed", n=16384, d=8192, v=131072, dtype="bf16", scale=90.5),
        # the embedding's gradient for the 1B layer's 4096 tokens
        dict(name="embed_grad_1b", op="embed_grad", n=4096, d=2048, v=32768, dtype="bf16",
             scale=45.25),
        # float32 training with an odd vocabulary: most of the time is the table's gradient
        dict(name="embed_grad_odd", op="embed_grad", n=8192, d=4096, v=49999, dtype="fp32",
             scale=1.0),
        # serving: the sampled tokens' log probabilities and 20 alternatives, 16 sequences
        dict(name="logprob_decode", op="logprob", n=16, v=131072, top=20, dtype="bf16", scale=1.0),
        # scoring a batch of 4096 tokens at a large vocabulary, with 5 alternatives
        dict(name="logprob_score", op="logprob", n=4096, v=131072, top=5, dtype="bf16", scale=1.25),
        # a training step's gradient of the loss, 1B layer's batch
        dict(name="logprob_grad_1b", op="logprob_grad", n=4096, v=32768, dtype="bf16", scale=1.0,
             entropy=False),
        # policy training with an entropy bonus, float32 logits, an odd vocabulary
        dict(name="logprob_grad_odd", op="logprob_grad", n=2000, v=49999, dtype="fp32", scale=0.8,
             entropy=True),
        # the layer's input saved in 8 bits and read back: a float32 batch
        dict(name="act8_fp32", op="act8", n=8192, d=4096, dtype="fp32"),
        # the same at the largest layer
        dict(name="act8_large", op="act8", n=16384, d=8192, dtype="bf16"),
        # the backward pass of the smallest layer: latency of the whole sequence
        dict(name="backward_act8_tiny", op="backward_act8", n=64, d=128, ff=512, tile=64, cap=8,
             b0=-1.645, dtype="fp32"),
        # the backward pass of the 1B layer
        dict(name="backward_act8_1b", op="backward_act8", n=4096, d=2048, ff=8192, tile=128, cap=4,
             b0=-2.326, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "logprob", "logprob_grad", "act8", "backward_act8"])
    dtype = rng.choice(["bf16", "fp32"])
    eb = 2 if dtype == "bf16" else 4
    if op in ("embed", "embed_grad"):
        n, d, v = _log_int(rng, 1, 16384), 8 * _log_int(rng, 16, 1024), _log_int(rng, 1000, 131072)
        v = min(v, (800 << 20) // (4 * d))
        return dict(op=op, n=n, d=d, v=v, dtype=dtype, scale=rng.choice([1.0, 32.0]))
    if op in ("logprob", "logprob_grad"):
        v = _log_int(rng, 1000, 131072)
        n = min(_log_int(rng, 1, 4096), (1 << 30) // (v * eb))
        case = dict(op=op, n=n, v=v, dtype=dtype, scale=rng.choice([1.0, 0.7, 1.4]))
        if op == "logprob":
            case["top"] = rng.choice([0, 1, 5, 20])
        else:
            case["entropy"] = rng.random() < 0.5
        return case
    if op == "act8":
        return dict(op=op, n=_log_int(rng, 1, 16384), d=8 * _log_int(rng, 16, 1024), dtype=dtype)
    tile, cap, b0 = rng.choice([(64, 8, -1.645), (128, 4, -2.326), (256, 8, -2.326)])
    return dict(op=op, n=_log_int(rng, 1, 4096), d=8 * _log_int(rng, 16, 256),
                ff=256 * _log_int(rng, 2, 32), tile=tile, cap=cap, b0=b0, dtype=dtype)


# ------------------------------------------------------------------ inputs
def _tokens(n, v, g):
    """Zipf-like token ids (the id's logarithm is uniform), 2% of them padding (-1)."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    t = (torch.exp(u * math.log(v + 1)).to(torch.int64) - 1).clamp_(0, v - 1)
    return torch.where(torch.rand(n, generator=g, device="cuda") < 0.02, -1, t)


def _hybrid(h, tile, cap):
    """h's hybrid form: per tile the first `cap` non-zeros and their places, and whole
    rows where a tile holds more."""
    n, ff = h.shape
    nt = ff // tile
    ht = h.view(n, nt, tile)
    nz = ht != 0
    over = (nz.sum(2) > cap).any(1)
    nz &= ~over[:, None, None]
    place = torch.where(nz, nz.cumsum(2) - 1, cap)
    values = torch.zeros((n, nt, cap + 1), dtype=h.dtype, device="cuda").scatter_(2, place, ht)
    column = torch.arange(tile, device="cuda", dtype=torch.uint8).expand(n, nt, tile)
    indices = torch.zeros((n, nt, cap + 1), dtype=torch.uint8, device="cuda")
    indices.scatter_(2, place, column)
    rows = over.nonzero()[:, 0]
    dense_rows = torch.zeros(n, dtype=torch.int32, device="cuda")
    dense_rows[:len(rows)] = rows.to(torch.int32)
    dense_values = torch.zeros((n, ff), dtype=h.dtype, device="cuda")
    dense_values[:len(rows)] = h[rows]
    return dict(values=values[:, :, :cap].contiguous(), indices=indices[:, :, :cap].contiguous(),
                counts=nz.sum(2).to(torch.uint8), dense_rows=dense_rows,
                dense_values=dense_values,
                n_dense=torch.tensor([len(rows)], dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, op, n = DTYPES[case["dtype"]], case["op"], case["n"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std).to(dt)

    s = dict(case)
    if op == "embed":
        s.update(table=normal(case["v"], case["d"], std=0.02), tokens=_tokens(n, case["v"], g))
    elif op == "embed_grad":
        s.update(dout=normal(n, case["d"]), tokens=_tokens(n, case["v"], g))
    elif op in ("logprob", "logprob_grad"):
        # a peaked distribution: a wide bulk, a few likely tokens per row, and the last
        # columns (a vocabulary padded to a round size) masked
        v = case["v"]
        logits = torch.randn((n, v), generator=g, device="cuda").mul_(2.0)
        likely = torch.randint(0, v, (n, 8), generator=g, device="cuda")
        logits.scatter_(1, likely, 8 + 3 * torch.randn((n, 8), generator=g, device="cuda"))
        targets = likely[:, 0].clone()
        logits[:, v - v // 100:] = -math.inf
        targets.clamp_(max=v - v // 100 - 1)
        # prompt tokens and padding carry no target
        targets[torch.rand(n, generator=g, device="cuda") < 0.03] = -100
        s.update(logits=logits.to(dt), targets=targets)
        if op == "logprob_grad":
            s.update(dlogp=-torch.rand(n, generator=g, device="cuda") / n,
                     dentropy=(-0.01 / n * torch.ones(n, device="cuda")
                               if case["entropy"] else None))
            # what the forward pass kept for this one
            z = s["logits"].float() * case["scale"]
            lse = torch.logsumexp(z, 1)
            z.sub_(lse[:, None])
            s.update(lse=lse, ent=-(z.exp().mul_(z)).nan_to_num_(0.0).sum(1))
    elif op == "act8":
        # token rows of unequal size
        scale = torch.exp(0.7 * torch.randn((n, 1), generator=g, device="cuda"))
        x = torch.randn((n, case["d"]), generator=g, device="cuda") * scale
        s.update(x=x.to(dt))
    else:
        d, ff = case["d"], case["ff"]
        x = normal(n, d)
        w_up_t, w_down = normal(ff, d, std=d ** -0.5), normal(ff, d, std=ff ** -0.5)
        h = torch.relu(x.float() @ w_up_t.float().t() + case["b0"]).to(dt)
        codes, scales = _codes(x)
        s.update(codes=codes, scales=scales, w_up_t=w_up_t, w_down=w_down, dy=normal(n, d),
                 hybrid=_hybrid(h, case["tile"], case["cap"]))
    return s


def _codes(x):
    """The 8-bit form of x [n, d]: one scale per row and block of columns, the largest
    magnitude over 127, and the nearest codes; rows of codes padded to 16."""
    n, d = x.shape
    nb = -(-d // BLOCK)
    f = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - d)).view(n, nb, BLOCK)
    a = f.abs().amax(2, keepdim=True)
    q = torch.round(f * 127 / torch.where(a > 0, a, 1.0))
    pitch = -(-d // 16) * 16
    return (q.view(n, -1)[:, :pitch].to(torch.int8).contiguous(), (a[:, :, 0] / 127).contiguous())


def _decoded(codes, scales, d):
    n, nb = scales.shape
    f = torch.nn.functional.pad(codes.float(), (0, nb * BLOCK - codes.shape[1]))
    return (f.view(n, nb, BLOCK) * scales[:, :, None]).view(n, -1)[:, :d]


# ------------------------------------------------------------------ one pass
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    from activation_sparse_transformer_amd import twell

    op = s["op"]
    # outputs and workspaces are made at the first pass and kept, as a training loop does
    if op == "embed":
        s["out"] = twell.twell_embed_forward(s["table"], s["tokens"], scale=s["scale"],
                                             out=s.get("out"))
        return s["out"]
    if op == "embed_grad":
        if "ws" not in s:
            s["ws"] = twell.embed_backward_workspace(s["n"], s["d"], s["v"], "cuda")
        s["out"] = twell.twell_embed_backward(s["dout"], s["tokens"], s["v"], scale=s["scale"],
                                              out=s.get("out"), workspace=s["ws"])
        return s["out"]
    if op == "logprob":
        if "ws" not in s:
            s["ws"] = twell.logprob_workspace(s["n"], s["v"], s["top"], s["logits"].dtype, "cuda")
        s["out"] = lp = twell.twell_logprob_forward(s["logits"], s["targets"], top=s["top"],
                                                    scale=s["scale"], out=s.get("out"),
                                                    workspace=s["ws"])
        return dict(logp=lp.logp, entropy=lp.entropy, lse=lp.lse, top_ids=lp.top_ids,
                    top_logp=lp.top_logp)
    if op == "logprob_grad":
        s["out"] = twell.twell_logprob_backward(s["logits"], s["targets"], s["lse"], s["ent"],
                                                s["dlogp"], s["dentropy"], scale=s["scale"],
                                                out=s.get("out"))
        return s["out"]
    if op == "act8":
        s["act"] = twell.twell_act8_pack(s["x"], out=s.get("act"))
        s["out"] = twell.twell_act8_unpack(s["act"], out=s.get("out"))
        return s["out"]
    if "act" not in s:
        s["act"] = twell.Act8(s["d"], s["w_up_t"].dtype, s["codes"], s["scales"])
        s["hy"] = twell.Hybrid(s["tile"], s["cap"], s["ff"], **s["hybrid"])
        s["ws"] = twell.backward_act8_workspace(s["hy"], s["d"])
    s["out"] = g = twell.ffn_sparse_backward_act8(s["act"], s["w_up_t"], s["w_down"], s["hy"],
                                                  s["dy"], out=s.get("out"), workspace=s["ws"])
    return dict(dx=g.dx, dw_up_t=g.dw_up_t, db_up=g.db_up, dw_down=g.dw_down)


def _run_plain(s):
    op = s["op"]
    if op == "embed":
        t = s["tokens"]
        rows = s["table"][t.clamp(min=0)].float() * s["scale"]
        return torch.where((t >= 0)[:, None], rows, 0.0).to(s["table"].dtype)
    if op == "embed_grad":
        t = s["tokens"]
        rows = torch.where((t >= 0)[:, None], s["dout"].float() * s["scale"], 0.0)
        out = torch.zeros((s["v"], s["d"]), device="cuda")
        return out.index_add_(0, t.clamp(min=0), rows)
    if op == "logprob":
        x, t = s["logits"].float(), s["targets"]
        z = x * s["scale"]
        m = z.amax(1, keepdim=True)
        e = torch.exp(z - m)
        total = e.sum(1, keepdim=True)
        lse = m + torch.log(total)
        lp = z - lse
        entropy = -torch.where(e > 0, e * lp, 0.0).sum(1) / total[:, 0]
        logp = torch.where(t >= 0, lp.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
        # alternatives by value, the lowest index first among equals: the float's order as
        # a whole number above, the column's below
        b = (x + 0.0).view(torch.int32).to(torch.int64)
        key = torch.where(b >= 0, b, -(b & 0x7fffffff)) * s["v"]
        key += torch.arange(s["v"] - 1, -1, -1, device="cuda")
        ids = s["v"] - 1 - key.topk(s["top"], dim=1).values % s["v"]
        return dict(logp=logp, entropy=entropy, lse=lse[:, 0], top_ids=ids.to(torch.int32),
                    top_logp=lp.gather(1, ids))
    if op == "logprob_grad":
        x, t = s["logits"].float(), s["targets"]
        lp = x * s["scale"] - s["lse"][:, None]
        p = torch.exp(lp)
        given = t >= 0
        gl = torch.where(given, s["dlogp"], 0.0)
        d = -gl[:, None] * p
        d.scatter_add_(1, t.clamp(min=0)[:, None], gl[:, None])
        if s["dentropy"] is not None:
            d -= torch.where(p > 0, p * (lp + s["ent"][:, None]), 0.0) * s["dentropy"][:, None]
        return (d * s["scale"]).to(s["logits"].dtype)
    if op == "act8":
        codes, scales = _codes(s["x"])
        return _decoded(codes, scales, s["d"]).to(s["x"].dtype)
    x, dy = _decoded(s["codes"], s["scales"], s["d"]), s["dy"].float()
    h = _dense(s["hybrid"], s["ff"], s["tile"], torch.float32)
    wu, wd = s["w_up_t"].float(), s["w_down"].float()
    dz = torch.where(h != 0, dy @ wd.t(), 0.0)
    return dict(dx=(dz @ wu).to(s["dy"].dtype), dw_up_t=dz.t() @ x, db_up=dz.sum(0),
                dw_down=h.t() @ dy)


def _dense(hy, ff, tile, dtype):
    """The dense h [n, ff] of a hybrid."""
    n, nt, cap = hy["values"].shape
    live = torch.arange(cap, device="cuda") < hy["counts"][:, :, None]
    h = torch.zeros((n, nt, tile), dtype=dtype, device="cuda")
    h.scatter_add_(2, hy["indices"].to(torch.int64),
                   torch.where(live, hy["values"], 0).to(dtype))
    stored = torch.arange(n, device="cuda") < hy["n_dense"]
    rows = torch.where(stored, hy["dense_rows"], 0).to(torch.int64)
    return h.view(n, ff).index_add_(0, rows, torch.where(stored[:, None], hy["dense_values"],
                                                         0).to(dtype))


# ------------------------------------------------------------------ what a pass cannot do without
def _distinct(n, v):
    """The expected number of distinct ids among n of _tokens."""
    p = np.log1p(1.0 / np.arange(1, v + 1)) / math.log(v + 1)
    return float(np.sum(-np.expm1(0.98 * n * np.log1p(-p))))


def work(case):
    op, n, eb = case["op"], case["n"], DTYPES[case["dtype"]].itemsize
    if op == "embed":
        d = case["d"]
        return dict(bytes=8 * n + (_distinct(n, case["v"]) + n) * d * eb, flops=n * d)
    if op == "embed_grad":
        d = case["d"]
        return dict(bytes=8 * n + n * d * eb + case["v"] * d * 4, flops=2 * n * d)
    if op == "logprob":
        v = case["v"]
        return dict(bytes=n * v * eb + n * (8 + 12 + 8 * case["top"]), flops=6 * n * v)
    if op == "logprob_grad":
        v = case["v"]
        return dict(bytes=2 * n * v * eb + n * (8 + 16), flops=(8 if case["entropy"] else 5) * n * v)
    if op == "act8":
        d = case["d"]
        return dict(bytes=2 * n * d * eb + 2 * (n * d + n * -(-d // BLOCK) * 4), flops=4 * n * d)
    # backward: h is active with the normal law's share of units, independently; a row is
    # dense when one of its tiles holds more than `cap`
    d, ff, tile, cap = case["d"], case["ff"], case["tile"], case["cap"]
    q = 0.5 * math.erfc(-case["b0"] / math.sqrt(2))
    fits = sum(math.comb(tile, k) * q ** k * (1 - q) ** (tile - k) for k in range(cap + 1))
    dense = n * (1 - fits ** (ff // tile))
    hybrid = n * (ff // tile) * (cap * (eb + 1) + 1) + dense * (ff * eb + 4)
    weights = 2 * ff * d * (eb + 4) + 4 * ff
    rows = n * d * (1 + 2 * eb) + n * -(-d // BLOCK) * 4
    return dict(bytes=hybrid + weights + rows, flops=8 * n * ff * q * d)


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        t = s["tokens"].cpu()
        rows = s["table"].cpu()[t.clamp(min=0)].double() * case["scale"]
        rows[t < 0] = 0
        return rows
    if op == "embed_grad":
        order = torch.argsort(s["tokens"], stable=True)
        out = torch.zeros((case["v"], case["d"]), dtype=torch.float64, device="cuda")
        order = order[s["tokens"][order] >= 0]
        out.index_put_((s["tokens"][order],), s["dout"][order].double() * case["scale"],
                       accumulate=True)
        return out
    if op == "logprob":
        parts = []
        for r in range(0, case["n"], 512):
            z = s["logits"][r:r + 512].double()
            by = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            z *= case["scale"]
            lse = torch.logsumexp(z, 1)
            lp = torch.log_softmax(z, 1)
            t = s["targets"][r:r + 512]
            picked = lp[torch.arange(len(t), device="cuda"), t.clamp(min=0)]
            picked[t < 0] = 0
            parts.append((picked, torch.special.entr(lp.exp()).sum(1), lse, by.to(torch.int32),
                          lp.gather(1, by)))
        logp, entropy, lse, ids, top = (torch.cat(p) for p in zip(*parts))
        return dict(logp=logp, entropy=entropy, lse=lse, top_ids=ids, top_logp=top)
    if op == "logprob_grad":
        out = torch.empty(s["logits"].shape, dtype=torch.float64, device="cuda")
        for r in range(0, case["n"], 512):
            rows = slice(r, r + 512)
            z = s["logits"][rows].double().requires_grad_(True)
            # the mask's columns apart: no gradient passes a place of probability zero
            lp = torch.log_softmax(z * case["scale"], 1)
            kept = torch.where(torch.isinf(z), 0.0, lp)
            t = s["targets"][rows]
            at = kept.gather(1, t.clamp(min=0)[:, None])[:, 0]
            loss = (at * s["dlogp"][rows].double() * (t >= 0)).sum()
            if s["dentropy"] is not None:
                loss = loss - ((kept.exp() * ~torch.isinf(z) * kept).sum(1)
                               * s["dentropy"][rows].double()).sum()
            out[rows] = torch.autograd.grad(loss, z)[0]
        return out
    if op == "act8":
        x = s["x"].double()
        out = torch.empty_like(x)
        for c in range(0, case["d"], BLOCK):
            f = x[:, c:c + BLOCK]
            step = f.abs().max(1, keepdim=True).values / 127
            out[:, c:c + BLOCK] = torch.round(f / step.clamp(min=1e-300)) * step
        return out
    hy = s["hybrid"]
    n, nt, cap = hy["values"].shape
    h = torch.zeros((n, case["ff"]), dtype=torch.float64, device="cuda")
    live = (torch.arange(cap, device="cuda") < hy["counts"][:, :, None]).nonzero(as_tuple=True)
    h[live[0], live[1] * case["tile"] + hy["indices"][live].to(torch.int64)] = \
        hy["values"][live].double()
    nd = int(hy["n_dense"])
    h[hy["dense_rows"][:nd].to(torch.int64)] = hy["dense_values"][:nd].double()
    steps = s["scales"].double().repeat_interleave(BLOCK, 1)[:, :case["d"]]
    x = s["codes"][:, :case["d"]].double() * steps
    dy, wu, wd = s["dy"].double(), s["w_up_t"].double(), s["w_down"].double()
    dz = (dy @ wd.t()) * (h != 0)
    return dict(dx=dz @ wu, dw_up_t=dz.t() @ x, db_up=dz.sum(0), dw_down=h.t() @ dy)
