"""AdamW in fp64 and the 8-bit form of its moments (E4M3 codes, one power-of-two scale per 32
elements, stochastic rounding), from their definitions.

`step` is the definition in fp64. `step32` does the same in fp32, one rounding per operation in the
order in which the header states them, and encodes the moments: what a kernel that rounds every
operation on its own has to give bit for bit.
"""
from __future__ import annotations

import math

import numpy as np

F = np.float32
M32 = 0xFFFFFFFF


def step(p, g, m, v, lr, beta1, beta2, eps, weight_decay, t, norm=None, max_norm=math.inf):
    """(p, m, v) after one step, fp64."""
    p, g, m, v = (np.asarray(a, np.float64) for a in (p, g, m, v))
    if norm is not None and norm > max_norm:
        g = g * (max_norm / norm)
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** t), v / (1 - beta2 ** t)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v


# ---- random bits --------------------------------------------------------------------------------

def mix(h):
    h = np.asarray(h, np.uint64) & M32
    h = h ^ (h >> 16)
    h = (h * 0x6A09E667) & M32
    h = h ^ (h >> 15)
    h = (h * 0xBB67AE85) & M32
    return h ^ (h >> 16)


def bits(seed: int, number: int, n: int, first: int = 0):
    """32 random bits for the elements first .. first + n - 1 of the call's tensor `number`."""
    i = np.arange(first, first + n, dtype=np.uint64)
    salt = mix((seed + number * 0x9E3779B1) & M32)
    return mix((i & M32) ^ mix((salt + (i >> 32)) & M32))


# ---- E4M3 runs ----------------------------------------------------------------------------------

def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes (4 exponent bits, bias 7, 3 mantissa bits; 0x7F: NaN)."""
    out = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        v = (8 + f) * 2.0 ** (e - 10) if e else f * 2.0 ** -9
        out[c] = (-v if c & 128 else v) if (c & 127) != 127 else math.nan
    return out


def decode(codes, scales) -> np.ndarray:
    """fp64 values of codes [n] with scales [ceil(n / 32)] (exact; 0xFF: NaN)."""
    s = np.where(np.asarray(scales) == 255, math.nan, 2.0 ** (np.asarray(scales, np.float64) - 127))
    return e4m3_values()[np.asarray(codes, np.uint8)] * np.repeat(s, 32)[:len(codes)]


def encode(x, u, positive: bool):
    """Codes and scales of fp32 values x with 16 random bits u each: scale 2^e the smallest power of two
    with amax <= 448 * 2^e; x / 2^e to floor(|x| / step + u / 2^16) steps (positive: at least one)."""
    n = len(x)
    pad = -n % 32
    x = np.concatenate([np.asarray(x, F), np.zeros(pad, F)]).reshape(-1, 32)
    u = np.concatenate([np.asarray(u, np.float64), np.zeros(pad)]).reshape(-1, 32)
    codes = np.zeros(x.shape, np.uint8)
    scales = np.zeros(len(x), np.uint8)
    table = {v: c for c, v in enumerate(e4m3_values()[:127])}
    for r in range(len(x)):
        amax = np.abs(x[r]).max()
        if not np.isfinite(amax):
            scales[r] = 255
            continue
        e = -127
        if amax > 0:
            e = math.frexp(float(amax))[1] - 9
            e += float(amax) > 448 * 2.0 ** e
            e = max(e, -127)
        scales[r] = e + 127
        for j in range(32):
            a = abs(float(x[r, j])) * 2.0 ** -e
            step_ = 2.0 ** (max(math.frexp(a)[1] - 1, -6) - 3) if a else 2.0 ** -9
            # (24 and 16 bits, at least 2^-40 away from an integer that they do not reach: fp64 is exact enough)
            k = math.floor(a / step_ + u[r, j] / 65536)
            if positive and a > 0:
                k = max(k, 1)
            codes[r, j] = table[k * step_] | (128 if np.signbit(x[r, j]) else 0)
    return codes.reshape(-1)[:n], scales


def bf16_random(x, u):
    """fp32 -> BF16 bits by adding 16 random bits below the kept ones."""
    b = np.asarray(x, F).view(np.uint32).astype(np.uint64)
    return (((b + np.asarray(u, np.uint64)) >> 16) & 0xFFFF).astype(np.uint16)


def step32(p, g, m, v, lr, beta1, beta2, eps, weight_decay, t, sumsq=None, max_norm=math.inf):
    """(p, m, v, sqrt(v)) in fp32, one rounding per operation."""
    p, g, m, v = (np.asarray(a, F) for a in (p, g, m, v))
    if sumsq is not None:
        norm = math.sqrt(sumsq)
        g = g * F(max_norm / norm if norm > max_norm else 1.0)
    m = m * F(beta1) + g * F(1 - beta1)
    v = v * F(beta2) + (g * g) * F(1 - beta2)
    r = np.sqrt(v)
    den = r * F(1 / math.sqrt(1 - beta2 ** t)) + F(eps)
    p = p * F(1 - lr * weight_decay) - (m / den) * F(lr / (1 - beta1 ** t))
    return p, m, v, r
