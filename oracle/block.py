"""Block-scaled FP8 (E4M3 codes, one fp32 scale for 128 values) and the products of sorted rows, from
their definitions.

`quantize_*` form the codes in fp32, one rounding an operation, as include/mok.h states them: what a
kernel has to give bit for bit. Products are fp64 sums of codes times scales, by group.
"""
from __future__ import annotations

import numpy as np

from .mx import e4m3_decode, e4m3_encode

F = np.float32
B = 128
TOP, LEAST = F(448), F(2.0 ** -100)


def up(n: int) -> int:
    return -(-n // B) * B


def padded_rows(rows: int, groups: int) -> int:
    return (rows + (B - 1) * groups) // B * B


def clean(offsets, rows: int):
    """Offsets within 0..rows that never fall."""
    return np.maximum.accumulate(np.clip(np.asarray(offsets, np.int64), 0, rows))


def columns(offsets):
    """Where each group's column codes begin, and end (padded)."""
    begin = np.concatenate([[0], np.cumsum([up(int(b - a)) for a, b in zip(offsets, offsets[1:])])])
    return [int(v) for v in begin]


def _encode(v):
    """E4M3 codes of fp32 values of at most 448 (and a rounding); NaN is 0x7F."""
    nan = np.isnan(v)
    c = e4m3_encode(np.where(nan, 0.0, v).astype(np.float64))
    return np.where(nan, 0x7F, c).astype(np.uint8)


def _blocks(x, axes):
    """(codes, scales) with one scale for all of `axes` of fp32 x."""
    with np.errstate(all="ignore"):
        amax = np.maximum(np.nanmax(np.where(np.isnan(x), F(0), np.abs(x)), axis=axes, keepdims=True), LEAST).astype(F)
        return _encode((x * (TOP / amax).astype(F)).astype(F)), (amax / TOP).astype(F)


def quantize_rows(x):
    """codes [R][up(K)], scales [up(K) / 128][R] of fp32 x [R][K]."""
    r, k = x.shape
    c, s = _blocks(np.pad(x.astype(F), ((0, 0), (0, up(k) - k))).reshape(r, up(k) // B, B), (2,))
    return c.reshape(r, up(k)), np.ascontiguousarray(s.reshape(r, up(k) // B).T)


def quantize_columns(x, offsets, codes, scales):
    """Fills column codes [K][P] and scales [P / 128][K] of the rows of each group."""
    for a, b, at in zip(offsets, offsets[1:], columns(offsets)):
        if b > a:
            c, s = quantize_rows(np.ascontiguousarray(x[a:b].T))
            codes[:, at:at + c.shape[1]] = c
            scales[at // B:at // B + s.shape[0]] = s


def quantize_weights(w):
    """codes [G][N][up(K)], scales [G][up(N) / 128][up(K) / 128] of fp32 w [G][N][K]."""
    g, n, k = w.shape
    p = np.pad(w.astype(F), ((0, 0), (0, up(n) - n), (0, up(k) - k))).reshape(g, up(n) // B, B, up(k) // B, B)
    c, s = _blocks(p, (2, 4))
    return c.reshape(g, up(n), up(k))[:, :n], s.reshape(g, up(n) // B, up(k) // B)


def values_rows(codes, scales):
    """fp64 values of codes [R][128 nb] with scales [nb][R]."""
    with np.errstate(all="ignore"):
        return e4m3_decode(codes) * np.repeat(scales.T.astype(np.float64), B, 1)


def values_weights(codes, scales):
    with np.errstate(all="ignore"):
        s = np.repeat(np.repeat(scales.astype(np.float64), B, 1)[:, :codes.shape[1]], B, 2)
        return e4m3_decode(codes) * s


def gemm(x, xs, w, ws, offsets, out):
    """out (fp64, in place) and, of each result, the sum of its terms' sizes and of its blocks' largest
    possible terms (128 times the largest of each operand's block)."""
    xv, wv = values_rows(x, xs), values_weights(w, ws)
    size, most = np.zeros_like(out), np.zeros_like(out)
    for g, (a, b) in enumerate(zip(offsets, offsets[1:])):
        out[a:b] = xv[a:b] @ wv[g].T
        size[a:b] = np.abs(xv[a:b]) @ np.abs(wv[g]).T
        for j in range(0, x.shape[1], B):
            most[a:b] += B * np.outer(np.abs(xv[a:b, j:j + B]).max(1, initial=0), np.abs(wv[g][:, j:j + B]).max(1, initial=0))
    return out, size, most


def wgrad(dy, dys, x, xs, offsets, dw):
    """Adds each group's dy^T x to dw (fp64, in place); returns it and the sum of the terms' sizes."""
    dv, xv = values_rows(dy, dys), values_rows(x, xs)
    size = np.abs(dw)
    at = columns(offsets)
    for g in range(len(offsets) - 1):
        d, v = dv[:, at[g]:at[g + 1]], xv[:, at[g]:at[g + 1]]
        dw[g] += d @ v.T
        size[g] += np.abs(d) @ np.abs(v).T
    return dw, size
