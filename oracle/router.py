"""The router in 64 bits: picks, probabilities, batch statistics and the gradient
of the logits, from their definitions (test infrastructure only)."""

from __future__ import annotations

import numpy as np

__all__ = ["route_forward", "route_objective", "route_backward"]


def _stats(x: np.ndarray):
    """softmax and logsumexp of each row; rows of nothing but -inf give zeros."""
    dead = np.isneginf(x).all(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        m = np.where(dead, 0.0, x.max(axis=1, keepdims=True))
        e = np.exp(x - m)
        z = e.sum(axis=1, keepdims=True)
        p = np.where(dead, 0.0, e / np.where(dead, 1.0, z))
        lse = np.where(dead, 0.0, m + np.log(np.where(dead, 1.0, z)))
    return p, lse


def _scores(x, sigmoid):
    p, lse = _stats(x)
    with np.errstate(over="ignore"):
        return (1.0 / (1.0 + np.exp(-x)) if sigmoid else p), p, lse


def route_forward(logits, k: int, sigmoid=False, renorm=False, scale=1.0):
    """dict(idx, prob, counts, losses) of logits [T, E] (any float array)."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    # NaN first, then larger first; a stable sort keeps ties in index order
    key = np.where(np.isnan(x), -np.inf, -x)
    order = np.lexsort((np.broadcast_to(np.arange(E), x.shape), key, ~np.isnan(x)), axis=1)
    idx = order[:, :k]
    s, _, lse = _scores(x, sigmoid)
    prob = np.take_along_axis(s, idx, 1)
    if renorm:
        tot = prob.sum(axis=1, keepdims=True)
        prob = np.where(tot == 0, 0.0, prob / np.where(tot == 0, 1.0, tot))
    counts = np.bincount(idx.reshape(-1), minlength=E)
    losses = np.zeros(2)
    if T:
        row = s.sum(axis=1, keepdims=True)
        share = s / np.where(row == 0, 1.0, row)
        losses[:] = E * np.dot(counts / (T * k), share.mean(axis=0)), (lse ** 2).mean()
    return dict(idx=idx.astype(np.int32), prob=scale * prob, counts=counts.astype(np.int32),
                losses=losses)


def route_objective(logits, idx, counts, dprob, sigmoid=False, renorm=False, scale=1.0, aux=0.0,
                    z=0.0) -> float:
    """<dprob, prob> + aux * balance loss + z * z loss with the picks and counts held fixed:
    the function whose gradient route_backward is."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    k = idx.shape[1]
    s, _, lse = _scores(x, sigmoid)
    prob = np.take_along_axis(s, idx.astype(np.int64), 1)
    if renorm:
        tot = prob.sum(axis=1, keepdims=True)
        prob = np.where(tot == 0, 0.0, prob / np.where(tot == 0, 1.0, tot))
    row = s.sum(axis=1, keepdims=True)
    share = s / np.where(row == 0, 1.0, row)
    balance = E * np.dot(counts / (T * k), share.mean(axis=0))
    return float((dprob * scale * prob).sum() + aux * balance + z * (lse ** 2).mean())


def route_backward(logits, idx, counts, dprob, sigmoid=False, renorm=False, scale=1.0, aux=0.0,
                   z=0.0):
    """(dlogits, mag): the gradient, and per element the sum of the magnitudes of the terms
    it is the signed sum of (the scale of its rounding error)."""
    x = np.asarray(logits, dtype=np.float64)
    T, E = x.shape
    k = idx.shape[1]
    idx = idx.astype(np.int64)
    s, p, lse = _scores(x, sigmoid)
    g = np.asarray(dprob, dtype=np.float64) * scale
    sel = np.take_along_axis(s, idx, 1)
    ga = np.abs(g)
    if renorm:
        tot = sel.sum(axis=1, keepdims=True)
        safe = np.where(tot == 0, np.inf, tot)
        share = sel / safe
        mean = (g * share).sum(axis=1, keepdims=True)
        ga = (ga + (ga * share).sum(axis=1, keepdims=True)) / safe
        g = (g - mean) / safe
    ds = np.zeros_like(x)
    dm = np.zeros_like(x)
    np.put_along_axis(ds, idx, g, 1)
    np.put_along_axis(dm, idx, ga, 1)
    load = E * counts / (T * k)
    row = s.sum(axis=1, keepdims=True)
    safe = np.where(row == 0, np.inf, row)
    mean = (load * s).sum(axis=1, keepdims=True) / safe
    ds = ds + aux / T * (load - mean) / safe
    dm = dm + abs(aux) / T * (load + mean) / safe
    if sigmoid:
        dx, mag = ds * s * (1 - s), dm * s
    else:
        dx = p * (ds - (ds * p).sum(axis=1, keepdims=True))
        mag = p * (dm + (dm * p).sum(axis=1, keepdims=True))
    dx = dx + z / T * 2 * lse * p
    mag = mag + abs(z) / T * 2 * np.abs(lse) * p
    return dx, mag
