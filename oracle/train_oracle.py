"""CPU oracle of the operators around the layer in a training step: 8-bit
activation checkpoints, the token embedding.  NumPy in float64, from the definitions."""
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
