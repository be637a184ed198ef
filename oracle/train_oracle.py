"""CPU oracle of the operators around the layer in a training step: 8-bit
activation checkpoints, the token embedding, log probabilities.  NumPy in
float64, from the definitions."""
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
