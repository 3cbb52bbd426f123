"""CPU oracle of the optimizer step (numpy): AdamW with fp32 or 8-bit states, stochastic rounding
by a hash, and the gradient norm.

With dtype float32 every operation is rounded as the kernel rounds it, so that results can be
compared bit for bit; with float64 it is the definition.
"""

from __future__ import annotations

import math

import numpy as np

CELL = 256
TOP = 448.0
AMAX_FLOOR = 2.0 ** -100
M32 = 0xFFFFFFFF


def mix(x):
    """Wellons' two-multiplication hash of 32 bits, on ints or uint64 arrays."""
    if isinstance(x, np.ndarray):
        x = x.astype(np.uint64) & M32
        x ^= x >> np.uint64(16)
        x = (x * np.uint64(0x7FEB352D)) & M32
        x ^= x >> np.uint64(15)
        x = (x * np.uint64(0x846CA68B)) & M32
        return x ^ (x >> np.uint64(16))
    x &= M32
    x ^= x >> 16
    x = (x * 0x7FEB352D) & M32
    x ^= x >> 15
    x = (x * 0x846CA68B) & M32
    return x ^ (x >> 16)


def noise(seed: int, step: int, position: int, n: int) -> np.ndarray:
    """32 random bits for each of a tensor's n elements."""
    key = mix(mix(mix(seed) + (step & M32)) + position)
    at = np.arange(n, dtype=np.uint64)
    cell = mix(np.uint64(key) + at // CELL)
    return mix(cell + at % CELL)


# values of the 256 E4M3 codes (0x7F and 0xFF: NaN)
def e4m3_table() -> np.ndarray:
    t = np.empty(256)
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        v = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        t[c] = math.nan if c & 127 == 127 else v
        if c & 128:
            t[c] = -t[c]
    return t


E4M3 = e4m3_table()


def round_code(y: np.ndarray, bits16: np.ndarray) -> np.ndarray:
    """Codes of y in [0, 448], up with the probability of the part cut off."""
    y = np.asarray(y)
    if y.dtype == np.float32:
        small = y < np.float32(2.0 ** -6)
        z = np.where(small, y + np.float32(2.0 ** -6), y).astype(np.float32)
        t = (z.view(np.uint32).astype(np.int64) + (bits16.astype(np.int64) << 4)) >> 20
        return np.minimum(t - np.where(small, 968, 960), 126)
    e = np.where(y > 0, np.maximum(np.frexp(y)[1] - 1, -6), -6)
    k = np.floor(y / 2.0 ** (e - 3.0) + bits16.astype(np.float64) / 65536)
    return np.minimum(np.where(e > -6, 8 * (e + 7) + k - 8, k), 126).astype(np.int64)


def _cells(x: np.ndarray) -> np.ndarray:
    n = x.size
    return np.concatenate([x, np.zeros(-n % CELL, x.dtype)]).reshape(-1, CELL)


def quantize(x: np.ndarray, bits16: np.ndarray, least_one: bool):
    """(codes, scales) of x by cells of 256."""
    dt = x.dtype.type
    n = x.size
    with np.errstate(all="ignore"):
        top = _cells(np.abs(x)).max(axis=1)  # NaN if any
        fine = np.isfinite(top)
        a = np.maximum(np.where(fine, top, 0), dt(AMAX_FLOOR)).astype(dt)
        inv = np.repeat(dt(TOP) * (dt(1) / a), CELL)[:n]
        y = np.where(np.repeat(fine, CELL)[:n], np.abs(x) * inv, 0).astype(dt)
    code = round_code(y, bits16)
    if least_one:
        code = np.where(x > 0, np.maximum(code, 1), code)
    code = np.where(x < 0, code | 128, code)
    code = np.where(np.repeat(fine, CELL)[:n], code, 0)
    return code.astype(np.uint8), np.where(fine, a * (dt(1) / dt(TOP)), np.nan).astype(dt)


def dequantize(codes: np.ndarray, scales: np.ndarray, dtype=np.float32) -> np.ndarray:
    return E4M3[codes].astype(dtype) * np.repeat(scales.astype(dtype), CELL)[:codes.size]


def power(beta: float, t: int) -> float:
    r, b = 1.0, beta
    while t > 0:
        if t & 1:
            r *= b
        b *= b
        t >>= 1
    return r


def step(w, g, m, v, *, lr, t, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, lr_scale=1.0,
         seed=0, position=0, grad_scale=1.0, bits=32, w_bf16=False, dtype=np.float32):
    """One step of one tensor. 8-bit states are passed and returned as (codes, scales). Returns
    (w, m, v); w is rounded to BF16 stochastically with w_bf16."""
    f = dtype
    per_step = lr / (1.0 - power(beta1, t))
    c1, c2 = f(per_step * lr_scale), f(1.0 / math.sqrt(1.0 - power(beta2, t)))
    kept = f(1.0 - lr * lr_scale * weight_decay)
    with np.errstate(all="ignore"):
        w, g = w.astype(f), g.astype(f) * f(grad_scale)
        if bits == 8:
            m = dequantize(*m, dtype=f)
            r = dequantize(*v, dtype=f)
            v = r * r
        m = m.astype(f) * f(beta1) + g * f(1.0 - beta1)
        v = v.astype(f) * f(beta2) + (g * g) * f(1.0 - beta2)
        r = np.sqrt(v)
        w = w * kept - (m * c1) / (r * c2 + f(eps))
    h = noise(seed, t, position, w.size)
    if bits == 8:
        m, v = quantize(m, h & np.uint64(0xFFFF), False), quantize(r, h >> np.uint64(16), True)
    if w_bf16:
        w = bf16_stochastic(w, mix(h + np.uint64(0x9E3779B9)) & np.uint64(0xFFFF))
    return w, m, v


def bf16_stochastic(w: np.ndarray, bits16: np.ndarray) -> np.ndarray:
    """BF16 values (in float32), up with the probability of the part cut off."""
    if w.dtype != np.float32:
        a = np.abs(w)
        e = np.maximum(np.frexp(a)[1] - 1, -126) - 7.0
        return np.sign(w) * np.floor(a / 2.0 ** e + bits16.astype(np.float64) / 65536) * 2.0 ** e
    b = w.view(np.uint32).astype(np.uint64)
    b = np.where(np.isfinite(w), b + bits16, b)
    out = (b & np.uint64(0xFFFF0000)).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(w), np.float32(np.nan), out)


def grad_norm(grads, max_norm: float = 0.0):
    """(norm, scale) in float64."""
    norm = math.sqrt(sum(float(np.square(x.astype(np.float64)).sum()) for x in grads))
    if not math.isfinite(norm):
        return norm, math.nan
    return norm, min(1.0, max_norm / (norm + 1e-6)) if max_norm > 0 else 1.0
