"""8-bit grouped linear layers in 64 bits (test infrastructure only): row codes and scales in the
fp32 arithmetic that defines them, products as exact integers, everything behind them in fp64."""

from __future__ import annotations

import numpy as np

__all__ = ["quantize_rows", "grouped_gemm"]

AMAX_FLOOR = np.float32(2.0 ** -100)


def quantize_rows(x):
    """(codes int8, scales fp32) of the rows of x (values exact in fp32), along the last axis."""
    x = np.asarray(x, dtype=np.float32)
    amax = np.abs(x).max(axis=-1, keepdims=True, initial=0)
    with np.errstate(invalid="ignore"):
        ok = np.isfinite(x).all(axis=-1, keepdims=True)
        a = np.maximum(np.where(ok, amax, np.float32(1)), AMAX_FLOOR)
        q = np.where(ok, np.rint(np.where(ok, x, 0) * (np.float32(127) / a)), 0)
        s = np.where(ok, a / np.float32(127), np.float32(np.nan))
    return q.astype(np.int8), s[..., 0].astype(np.float32)


def grouped_gemm(Aq, As, Wq, Ws, offsets, alpha=0.0, prob=None):
    """C in fp64 [R, N] (alpha 0) or [R, N/2] (gated with g * sigmoid(alpha g) * u), zero on rows
    no expert owns."""
    R, N = Aq.shape[0], Wq.shape[1]
    v = np.zeros((R, N))
    for e in range(Wq.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        acc = Aq[lo:hi].astype(np.int64) @ Wq[e].astype(np.int64).T
        with np.errstate(invalid="ignore"):
            v[lo:hi] = acc * As[lo:hi, None].astype(np.float64) * Ws[e].astype(np.float64)
    if not alpha:
        return v
    g, u = v[:, :N // 2], v[:, N // 2:]
    with np.errstate(over="ignore"):
        y = g / (1.0 + np.exp(-alpha * g)) * u
    return y if prob is None else y * np.asarray(prob, dtype=np.float64)[:, None]
