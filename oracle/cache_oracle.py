"""Float64 oracle of the paged cache: block means, routing of single queries, their attention
over kept blocks, and eviction by accumulated weight. One sequence and one key head at a time,
over that sequence's tokens in order (keys and values [n, d]); paging is the caller's."""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64


def block_means(k: np.ndarray) -> np.ndarray:
    """float32 [ceil(n / 64), d]: means of consecutive blocks of keys, rounded once."""
    n = k.shape[0]
    return np.array([k[i:i + BLOCK].astype(np.float64).sum(0) / min(BLOCK, n - i) for i in range(0, n, BLOCK)],
                    dtype=np.float64).reshape(-1, k.shape[1]).astype(np.float32)


def route(q: np.ndarray, means: np.ndarray, p: float, k_floor: int, n_recent: int, scale=None) -> np.ndarray:
    """Kept blocks (ascending) for the query heads q [G, d] of one key head."""
    nB = means.shape[0]
    if nB == 0:
        return np.zeros(0, dtype=np.int64)
    if p >= 1.0:
        return np.arange(nB)
    scale = 1.0 / math.sqrt(q.shape[1]) if scale is None else scale
    s = scale * (q.astype(np.float64) @ means.astype(np.float64).T)
    e = np.exp(s - s.max(1, keepdims=True))
    share = (e / e.sum(1, keepdims=True)).mean(0)
    order = np.lexsort((np.arange(nB), -share))
    total, count = 0.0, 0
    while count < nB and (total < p or count < k_floor):
        total += share[order[count]]
        count += 1
    return np.union1d(order[:count], np.arange(max(0, nB - n_recent), nB)).astype(np.int64)


def tokens_of(blocks: np.ndarray, n: int) -> np.ndarray:
    at = (np.asarray(blocks, dtype=np.int64)[:, None] * BLOCK + np.arange(BLOCK)).ravel()
    return at[at < n]


def attention(q: np.ndarray, k: np.ndarray, v: np.ndarray, blocks: np.ndarray, scale=None):
    """O [G, d], lse [G] and the weights [G, tokens] over the tokens of the kept blocks."""
    scale = 1.0 / math.sqrt(q.shape[1]) if scale is None else scale
    at = tokens_of(blocks, k.shape[0])
    if at.size == 0:
        return np.zeros((q.shape[0], v.shape[1])), np.full(q.shape[0], -np.inf), np.zeros((q.shape[0], 0)), at
    s = scale * (q.astype(np.float64) @ k[at].astype(np.float64).T)
    m = s.max(1, keepdims=True)
    z = np.exp(s - m).sum(1, keepdims=True)
    w = np.exp(s - m) / z
    return w @ v[at].astype(np.float64), (m + np.log(z))[:, 0], w, at


def evict(mass: np.ndarray, keep: int, n_sink: int, n_recent: int) -> np.ndarray:
    """Kept positions (ascending) of a sequence whose tokens have these weights."""
    n = mass.shape[0]
    if n <= keep:
        return np.arange(n)
    lo, hi = n_sink, n - n_recent
    w = np.where(np.isnan(mass[lo:hi]), -np.inf, mass[lo:hi].astype(np.float64))
    nan_last = np.isnan(mass[lo:hi])
    best = lo + np.lexsort((np.arange(hi - lo), nan_last, -w))[:keep - n_sink - n_recent]
    return np.concatenate([np.arange(lo), np.sort(best), np.arange(hi, n)])
