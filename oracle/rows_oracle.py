"""Float64 oracle of the operators on rows of vocabulary logits: filtered
sampling, the filtered speculative accept, top logits and distillation.

One row at a time, straight from the definitions (numpy); test infrastructure
only, sharing no code with the CUDA path.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np


def row_order(z) -> np.ndarray:
    """Unmasked entries (not NaN, not -inf) by descending value, ascending index."""
    z = np.asarray(z, np.float64)
    ids = np.nonzero(~np.isnan(z) & (z > -np.inf))[0]
    return ids[np.lexsort((ids, -z[ids]))]


def filtered(z, T: float, top_k: int = 0, top_p: float = 1.0, min_p: float = 0.0):
    """Kept token ids in order and their probabilities; empty if nothing counts."""
    z = np.asarray(z, np.float64)
    ids = row_order(z)
    if ids.size == 0:
        return ids, np.zeros(0)
    if T == 0:
        return ids[:1], np.ones(1)
    if top_k > 0:
        ids = ids[:top_k]
    m = z[ids[0]]
    with np.errstate(invalid="ignore"):
        w = np.where(z[ids] == m, 1.0, np.exp((z[ids] - m) / T))
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep = before < top_p * w.sum()
        keep[0] = True
        ids, w = ids[keep], w[keep]
    if min_p > 0:
        keep = z[ids] >= m + T * math.log(min_p)
        ids, w = ids[keep], w[keep]
    return ids, w / w.sum()


def gumbel_draw(ids, p, u, drop: Optional[int] = None):
    """(token, gap to the runner-up); (-1, inf) when nothing is left."""
    keep = ids != drop if drop is not None else np.ones(ids.size, bool)
    ids, p = ids[keep], p[keep]
    if ids.size == 0:
        return -1, math.inf
    with np.errstate(divide="ignore"):
        s = np.log(p) - np.log(-np.log(np.asarray(u, np.float64)[ids]))
    best = s.max()
    tok = int(ids[s == best].min())
    rest = s[ids != tok]
    return tok, float(best - rest.max()) if rest.size else math.inf


def sample(z, T, u, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log-probability, gap)."""
    ids, p = filtered(z, T, top_k, top_p, min_p)
    if ids.size == 0:
        return -1, -math.inf, math.inf
    if T == 0:
        return int(ids[0]), 0.0, math.inf
    tok, gap = gumbel_draw(ids, p, u)
    return tok, float(np.log(p[ids == tok][0])), gap


def verify_accept_filtered(z, draft, T, u_accept, u_sample, top_k=0, top_p=1.0, min_p=0.0):
    """z [R][V]; returns (n, corr, emitted, next_tok)."""
    R, D = len(z), len(draft)
    n, drop = 0, None
    while n < D:
        ids, p = filtered(z[n], T, top_k, top_p, min_p)
        hit = p[ids == draft[n]]
        if not (hit.size and u_accept[n] < hit[0]):
            drop = int(draft[n])
            break
        n += 1
    corr = -1
    if n < R:
        ids, p = filtered(z[n], T, top_k, top_p, min_p)
        corr = gumbel_draw(ids, p, u_sample, drop)[0]
    emitted = [int(x) for x in draft[:n]] + ([corr] if n < R else [])
    emitted += [-1] * (R - len(emitted))
    nxt = corr if corr >= 0 else (int(draft[n - 1]) if n else -1)
    return n, corr, np.asarray(emitted, np.int32), nxt


def top_logits(z, K: int, T: float = 1.0):
    """(values [K], indices [K], log-sum-exp of z / T)."""
    z = np.asarray(z, np.float64)
    ids = row_order(z)
    val, idx = np.full(K, -np.inf), np.full(K, -1, np.int32)
    k = min(K, ids.size)
    idx[:k], val[:k] = ids[:k], z[ids[:k]]
    if ids.size == 0:
        return val, idx, -math.inf
    m = z[ids[0]]
    return val, idx, float(m / T + math.log(np.exp((z[ids] - m) / T).sum()))


def _lse(x):
    x = np.asarray(x, np.float64)
    m = x.max() if x.size else -np.inf
    return -math.inf if m == -np.inf else float(m + math.log(np.exp(x - m).sum()))


def distill(z, t_val, t_idx, T: float = 1.0, t_lse: Optional[float] = None, weight: float = 1.0):
    """(loss, gradient [V]) of one row."""
    z = np.asarray(z, np.float64)
    V = z.size
    t_val, t_idx = np.asarray(t_val, np.float64), np.asarray(t_idx)
    listed = t_idx != -1
    ids = t_idx[listed]
    if np.any((ids < 0) | (ids >= V)) or np.unique(ids).size != ids.size:
        return math.nan, np.zeros(V)
    t = t_val[listed] / T
    if weight == 0:
        return 0.0, np.zeros(V)
    if np.any(np.isnan(t) | (t == np.inf)):
        return math.nan, np.zeros(V)
    if not np.any(t > -np.inf):
        return 0.0, np.zeros(V)
    if t_lse is not None and not math.isfinite(t_lse):
        return math.nan, np.zeros(V)
    m = z.max() if np.isfinite(z.max()) else 0.0  # softmax does not see a shift; sums keep their precision
    zt = (z - m) / T
    L = _lse(zt)
    if t_lse is None:
        t = (t_val[listed] - t_val[listed].max()) / T
    lp = t - (_lse(t) if t_lse is None else float(t_lse))
    p = np.exp(lp)
    if np.any(p > 256):
        return math.nan, np.zeros(V)
    on = p > 0
    loss = float((p[on] * (lp[on] - (zt[ids][on] - L))).sum())
    outside = np.ones(V, bool)
    outside[ids] = False
    pr = 0.0 if t_lse is None else max(0.0, 1.0 - p.sum())
    Lr = _lse(zt[outside])
    if t_lse is not None and pr <= 2.0 ** -20 * (1 + abs(t_lse)) and Lr - L < -126 * math.log(2):
        pr = 0.0  # no more than t_lse's rounding, over tokens that the student leaves out
    if pr > 0:
        loss += pr * (math.log(pr) - (Lr - L))
    P = p.sum() + pr
    grad = P * np.exp(zt - L)
    grad[ids] -= p
    if pr > 0 and Lr > -np.inf:
        w = np.exp(zt[outside] - zt[outside].max())
        grad[outside] -= pr * w / w.sum()
    return weight * loss, grad * (weight / T)
