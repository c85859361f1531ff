"""Float64 gradient of block-sparse attention, from the formulas.

With P = softmax over a row's kept keys of scale q.k, O = P V and a loss whose gradient with
respect to O is dO:  dP = dO V^T, dS = P (dP - rowsum(P dP)), dQ = scale dS K,
dK = scale dS^T Q, dV = P^T dO."""
from __future__ import annotations

import math

import numpy as np


def token_mask(keep_blocks: np.ndarray, N: int, block: int = 64) -> np.ndarray:
    """[nB, nB] kept blocks -> [N, N] visible (query, key) pairs."""
    at = np.arange(N) // block
    return keep_blocks[at][:, at]


def attention(q, k, v, seen, scale=None):
    """One head: O, lse, P for q, k, v [N, d] and the visible pairs; rows that see nothing give 0, -inf, 0."""
    scale = 1.0 / math.sqrt(q.shape[1]) if scale is None else scale
    s = np.where(seen, scale * (q @ k.T), -np.inf)
    m = np.max(s, axis=1, keepdims=True)
    e = np.where(seen, np.exp(s - np.where(np.isfinite(m), m, 0.0)), 0.0)
    z = e.sum(1, keepdims=True)
    p = np.divide(e, z, out=np.zeros_like(e), where=z > 0)
    with np.errstate(divide="ignore"):
        lse = np.where(z[:, 0] > 0, np.where(np.isfinite(m[:, 0]), m[:, 0], 0.0) + np.log(z[:, 0]), -np.inf)
    return p @ v, lse, p


def attention_grad(q, k, v, do, seen, scale=None):
    """One head: (dQ, dK, dV), each [N, d]."""
    scale = 1.0 / math.sqrt(q.shape[1]) if scale is None else scale
    _, _, p = attention(q, k, v, seen, scale)
    dp = do @ v.T
    ds = p * (dp - (p * dp).sum(1, keepdims=True))
    return scale * ds @ k, scale * ds.T @ q, p.T @ do
