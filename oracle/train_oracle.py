"""CPU oracle of the operators around the layer in a training step: 8-bit
activation checkpoints, the token embedding, log probabilities, the norms around
the layer, the output head, orthogonalised updates.  NumPy in float64, from the definitions."""
from __future__ import annotations

import numpy as np

ACT8_BLOCK = 128


def act8_quotients(x: np.ndarray):
    """x * 127 / a per element in float64, and a [N, blocks]: a is the largest
    magnitude of the row's block of columns (a zero block's quotients are 0)."""
    n, d = x.shape
    nb = -(-d // ACT8_BLOCK)
    q = np.zeros((n, d))
    a = np.zeros((n, nb))
    for b in range(nb):
        cols = slice(b * ACT8_BLOCK, min(d, (b + 1) * ACT8_BLOCK))
        top = np.abs(x[:, cols]).max(axis=1) if n else np.zeros(0)
        a[:, b] = top
        q[:, cols] = x[:, cols] * 127.0 / np.where(top > 0, top, 1.0)[:, None]
    return q, a


def act8_decode(codes: np.ndarray, scales: np.ndarray, d: int) -> np.ndarray:
    """code * scale in float64 for codes [N, >= d], scales [N, blocks]."""
    per_column = np.repeat(scales.astype(np.float64), ACT8_BLOCK, axis=1)[:, :d]
    return codes[:, :d].astype(np.float64) * per_column


def embed(table: np.ndarray, tokens: np.ndarray, scale: float) -> np.ndarray:
    """scale * table[tokens] in float64; ids outside the table give zeros."""
    ok = (tokens >= 0) & (tokens < len(table))
    out = np.zeros((len(tokens), table.shape[1]))
    out[ok] = table[tokens[ok]] * scale
    return out


def embed_grad(dout: np.ndarray, tokens: np.ndarray, vocab: int, scale: float) -> np.ndarray:
    """scale * the sums of dout's rows per id, in float64."""
    out = np.zeros((vocab, dout.shape[1]))
    ok = (tokens >= 0) & (tokens < vocab)
    np.add.at(out, tokens[ok], dout[ok])
    return out * scale


def logprob(x: np.ndarray, targets: np.ndarray, scale: float, top: int):
    """logp, entropy, lse, ids and log probabilities of the alternatives for logits x
    [N, V] in float64, row by row from the definitions."""
    n, v = x.shape
    logp, entropy, lse = np.zeros(n), np.zeros(n), np.zeros(n)
    ids, tops = np.full((n, top), -1), np.full((n, top), -np.inf)
    for r in range(n):
        live = x[r] != -np.inf
        if np.isnan(x[r]).any() or (x[r] == np.inf).any():
            logp[r] = entropy[r] = lse[r] = np.nan
        elif not live.any():
            lse[r] = logp[r] = -np.inf
        else:
            z = x[r] * scale
            m = z.max()
            ln_s = np.log(np.exp(z - m).sum())
            lse[r] = m + ln_s
            lp = (z[live] - m) - ln_s
            entropy[r] = -(np.exp(lp) * lp).sum()
            if 0 <= targets[r] < v:
                logp[r] = (z[targets[r]] - m) - ln_s
        if not 0 <= targets[r] < v:
            logp[r] = 0.0
        order = sorted((j for j in np.nonzero(live & ~np.isnan(x[r]))[0]),
                       key=lambda j: (-x[r, j], j))[:top]
        ids[r, :len(order)] = order
        if np.isnan(lse[r]):
            tops[r, :len(order)] = np.nan
        elif order:
            tops[r, :len(order)] = (x[r, order] * scale - m) - ln_s
    return logp, entropy, lse, ids, tops


def logprob_grad(x, targets, scale, dlogp, dentropy):
    """The gradient of sum(dlogp * logp + dentropy * entropy) in float64."""
    n, v = x.shape
    out = np.zeros((n, v))
    for r in range(n):
        live = x[r] != -np.inf
        if not live.any():
            continue
        z = x[r] * scale
        lp = (z[live] - z.max()) - np.log(np.exp(z - z.max()).sum())
        p = np.exp(lp)
        g = dlogp[r] if 0 <= targets[r] < v else 0.0
        d = -g * p - dentropy[r] * p * (lp - (p * lp).sum())
        out[r, live] = d
        if g:
            out[r, targets[r]] += g
    return out * scale


def norm(residual, y, w_post, gate, w_pre, alpha: float, eps: float):
    """(r', x) of the norms around the layer; y, the weights or x may be None."""
    r = residual
    if y is not None:
        u = y
        if w_post is not None:
            u = y / np.sqrt((y * y).mean(axis=1, keepdims=True) + eps) * w_post
        r = alpha * residual + (u if gate is None else gate * u)
    x = None
    if w_pre is not None:
        x = r / np.sqrt((r * r).mean(axis=1, keepdims=True) + eps) * w_pre
    return r, x


def norm_grad(residual_out, y, w_post, gate, w_pre, dr, dx, alpha: float, eps: float) -> dict:
    """Gradients of sum(dr * r' + dx * x) from r' and y, with the size of what each sum adds up
    ("of_" names: the same formulas over magnitudes), by which float32 results are judged."""
    n, d = residual_out.shape
    g = np.zeros((n, d)) if dr is None else dr
    of_g = np.abs(g)
    out = {}
    if w_pre is not None:
        rstd = 1 / np.sqrt((residual_out ** 2).mean(axis=1, keepdims=True) + eps)
        rn, p = residual_out * rstd, dx * w_pre
        g = g + rstd * (p - rn * (p * rn).mean(axis=1, keepdims=True))
        of_g = of_g + rstd * (np.abs(p) + np.abs(rn) * np.abs(p * rn).mean(axis=1, keepdims=True))
        out.update(dw_pre=(dx * rn).sum(axis=0), of_dw_pre=np.abs(dx * rn).sum(axis=0))
    out.update(d_residual=alpha * g, of_d_residual=np.abs(alpha) * of_g)
    if y is not None:
        w = np.ones(d) if gate is None else gate
        q, of_q, yn = g * w, of_g * np.abs(w), y
        dy, of_dy = q, of_q
        if w_post is not None:
            q, of_q = q * w_post, of_q * np.abs(w_post)
            ystd = 1 / np.sqrt((y * y).mean(axis=1, keepdims=True) + eps)
            yn = y * ystd
            dy = ystd * (q - yn * (q * yn).mean(axis=1, keepdims=True))
            of_dy = ystd * (of_q + np.abs(yn) * (of_q * np.abs(yn)).mean(axis=1, keepdims=True))
        out.update(dy=dy, of_dy=of_dy)
        total, of_total = (g * yn).sum(axis=0), (of_g * np.abs(yn)).sum(axis=0)
        if w_post is not None:
            out.update(dw_post=total * w, of_dw_post=of_total * np.abs(w))
        if gate is not None:
            by = np.ones(d) if w_post is None else w_post
            out.update(dgate=total * by, of_dgate=of_total * np.abs(by))
    return out


def head_logprob(x, w, targets, scale: float):
    """(logp, lse, stats, z) of targets under softmax(z), z = scale * x w^T; a target outside the
    vocabulary has logp 0."""
    z = scale * (x @ w.T)
    m = z.max(axis=1)
    with np.errstate(invalid="ignore", divide="ignore"):
        s = np.where(np.isneginf(m), 0.0, np.exp(z - m[:, None]).sum(axis=1))
        lse = np.where(np.isneginf(m), -np.inf, m + np.log(s))
    ok = (targets >= 0) & (targets < len(w))
    at = z[np.arange(len(z)), np.where(ok, targets, 0)]
    with np.errstate(invalid="ignore"):
        logp = np.where(ok, np.where(np.isneginf(lse), -np.inf, at - lse), 0.0)
    return logp, lse, np.stack([m, s], axis=1), z


def head_logprob_grad(x, w, targets, dlogp, scale: float):
    """(dx, dw, dl) of sum(dlogp * logp); rows without a target take no part."""
    ok = (targets >= 0) & (targets < len(w))
    dl = np.zeros((len(x), len(w)))
    logp, lse, _, z = head_logprob(x[ok], w, targets[ok], scale)
    live = ~np.isneginf(lse)
    with np.errstate(invalid="ignore"):
        p = np.where(live[:, None], np.exp(z - lse[:, None]), 0.0)
    d = -p
    d[np.arange(len(d)), targets[ok]] += 1
    dl[ok] = np.where(live[:, None], d, 0.0) * (scale * dlogp[ok])[:, None]
    x = np.where(ok[:, None], x, 0.0)
    return dl @ w, dl.T @ x, dl


def orthogonalize(m, steps: int, coefficients, eps: float, scale: float):
    """scale * U f(S) V^T of m / (|m| + eps) = U S V^T, f the steps' polynomial iterated on the
    singular values."""
    a, b, c = coefficients
    u, s, vt = np.linalg.svd(m / (np.sqrt((m * m).sum()) + eps), full_matrices=False)
    for _ in range(steps):
        s = a * s + b * s ** 3 + c * s ** 5
    return scale * (u * s) @ vt
