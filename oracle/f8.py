"""CPU oracle of the E4M3 products with scales per block of 128 (numpy, float64 but for the codes
and scales, which are 8-bit and 32-bit numbers and decided in float32 as the library does).

Tensor cores, fp32 sums and BF16 results are not modelled; `terms` returns the sums of the terms'
magnitudes that a test's tolerance is made of.
"""

from __future__ import annotations

import numpy as np

from .adamw import E4M3

BLOCK = 128
TOP = np.float32(448.0)
AMAX_FLOOR = np.float32(2.0 ** -100)


def encode(y: np.ndarray) -> np.ndarray:
    """E4M3 codes of float32 values, to nearest even, saturating."""
    a = np.minimum(np.abs(y.astype(np.float64)), 448.0)
    e = np.where(a > 0, np.maximum(np.frexp(a)[1] - 1, -6), -6)
    k = np.rint(a / 2.0 ** (e - 3.0))
    code = np.where(e > -6, 8 * (e + 7) + k - 8, k).astype(np.int64)
    return np.where(np.signbit(y), code | 128, code).astype(np.uint8)


def _scale(top):
    fine = np.isfinite(top)
    a = np.maximum(np.where(fine, top, 0).astype(np.float32), AMAX_FLOOR)
    inv = np.where(fine, (np.float32(1) / a) * TOP, 0).astype(np.float32)
    return inv, np.where(fine, a * (np.float32(1) / TOP), np.nan).astype(np.float32)


def quantize_rows(x: np.ndarray):
    """(codes [R][K] uint8, scales [ceil(K / 128)][R] float32) of float32 rows."""
    x = x.astype(np.float32)
    R, K = x.shape
    Q = np.zeros((R, K), np.uint8)
    S = np.zeros((-(-K // BLOCK), R), np.float32)
    with np.errstate(invalid="ignore"):
        for b in range(S.shape[0]):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            inv, S[b] = _scale(np.abs(part).max(axis=1))
            y = np.where(inv[:, None] > 0, part * inv[:, None], np.float32(0))
            Q[:, b * BLOCK:(b + 1) * BLOCK] = encode(y)
    return Q, S


def quantize_weight(W: np.ndarray):
    """(codes [E][N][K], scales [E][ceil(N / 128)][ceil(K / 128)]) of float32 weights."""
    W = W.astype(np.float32)
    E, N, K = W.shape
    Q = np.zeros(W.shape, np.uint8)
    S = np.zeros((E, -(-N // BLOCK), -(-K // BLOCK)), np.float32)
    with np.errstate(invalid="ignore"):
        for e in range(E):
            for i in range(S.shape[1]):
                for j in range(S.shape[2]):
                    at = (e, slice(i * BLOCK, (i + 1) * BLOCK), slice(j * BLOCK, (j + 1) * BLOCK))
                    inv, S[e, i, j] = _scale(np.abs(W[at]).max())
                    y = np.where(inv > 0, W[at] * inv, np.float32(0))
                    Q[at] = encode(y)
    return Q, S


def rows_value(Q, S):
    return E4M3[Q] * np.repeat(S.astype(np.float64).T, BLOCK, axis=1)[:, :Q.shape[1]]


def weight_value(Q, S):
    s = np.repeat(np.repeat(S.astype(np.float64), BLOCK, axis=-2), BLOCK, axis=-1)
    return E4M3[Q] * s[..., :Q.shape[-2], :Q.shape[-1]]


def product(Q, S, Wq, Ws, offsets, grad=False):
    """(sums, terms) [R][N] (grad: [R][K]): each row against its expert's weight; zero rows
    behind the last expert's. Codes are uint8."""
    R = Q.shape[0]
    x = rows_value(Q, S)
    E, N, K = Wq.shape
    y = np.zeros((R, K if grad else N))
    mag = np.zeros_like(y)
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if hi > lo:
            w = weight_value(Wq[e], Ws[e])
            w = w if grad else w.T
            y[lo:hi] = x[lo:hi] @ w
            mag[lo:hi] = np.abs(x[lo:hi]) @ np.abs(w)
    return y, mag


def sigmoid(x):
    e = np.exp(-np.abs(x))  # no cancellation on either side
    return np.where(x < 0, e, 1.0) / (1.0 + e)


def glu(g, u, alpha=1.0):
    return g * sigmoid(alpha * g) * u


def glu_bwd(acc, g, u, alpha=1.0, scale=None):
    """(dg, du, acc * act(g) u) for a gradient acc of the activation's output."""
    d = acc if scale is None else acc * scale[:, None]
    s = sigmoid(alpha * g)
    return d * u * s * (1 + alpha * g * (1 - s)), d * g * s, acc * g * s * u
