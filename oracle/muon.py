"""Muon in fp64, and with the roundings that a kernel makes.

`orthogonalize` is the definition. `rounded` does the same steps with X, A = X X^T and B = b A + c A A
rounded to fp16 where they are operands, but for A's and B's diagonals, sums exact: how far it is from the definition is
what those roundings cost. Matrices of up to 32 rows or columns are not rounded.
"""
from __future__ import annotations

import math

import numpy as np

JORDAN = (3.4445, -4.7750, 2.0315)


def orthogonalize(u, eps=1e-7, steps=5, coefficients=None):
    u = np.asarray(u, np.float64)
    if u.shape[0] > u.shape[1]:
        return orthogonalize(u.T, eps, steps, coefficients).T
    x = u / (math.sqrt(float((u * u).sum())) + eps)
    for a, b, c in coefficients or [JORDAN] * steps:
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


def _half(x):
    return x.astype(np.float16).astype(np.float64)


def _nineteen(x):
    """fp16, and a byte of 256ths of its last place."""
    h = _half(x)
    _, e = np.frexp(np.where(h == 0, 1.0, h))
    place = np.exp2(np.maximum(np.where(h == 0, -99, e), -13) - 11.0)   # (2^-24 below 2^-14)
    return h + np.clip(np.rint((x - h) / place * 256), -128, 127) / 256 * place


def _half_beside(x):
    """fp16, but on the diagonal."""
    d = np.diag(np.diag(x))
    return _half(x - d) + d


def rounded(u, eps=1e-7, steps=5, coefficients=None, small=False):
    """`small`: X kept in fp32; else in 19 bits."""
    u = np.asarray(u, np.float64)
    if min(u.shape) <= 32:
        return orthogonalize(u, eps, steps, coefficients)
    if u.shape[0] > u.shape[1]:
        return rounded(u.T, eps, steps, coefficients, small).T
    n, scale = u.shape[1], 1.0
    while n > 1:
        n, scale = n >> 2, scale * 2
    keep = (lambda x: x.astype(np.float32).astype(np.float64)) if small else _nineteen
    x = keep(u * (scale / (math.sqrt(float((u * u).sum())) + eps)))
    for a, b, c in coefficients or [JORDAN] * steps:
        h = _half(x)
        g = _half_beside(h @ h.T / scale ** 2)
        x = keep(a * x + _half_beside(b * g + c * (g @ g)) @ h)
    return x / scale


def adjustment(rule, rows, cols):
    return {"rms": 0.2 * math.sqrt(max(rows, cols)), "spectral": math.sqrt(max(1.0, rows / cols)), "none": 1.0}[rule]


def step(p, g, m, lr, momentum=0.95, nesterov=True, weight_decay=0.0, eps=1e-7, adjust="rms", steps=5,
         coefficients=None, norm=None, max_norm=math.inf):
    """(p, m, u) of one matrix after one step, u what was orthogonalised."""
    p, g, m = (np.asarray(a, np.float64) for a in (p, g, m))
    if norm is not None and norm > max_norm:
        g = g * (max_norm / norm)
    m = momentum * m + g
    u = g + momentum * m if nesterov else m
    o = orthogonalize(u, eps, steps, coefficients)
    return p - lr * weight_decay * p - lr * adjustment(adjust, *p.shape) * o, m, u
