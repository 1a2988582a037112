"""Buffer ownership for linear maps of sorted rows in block-scaled FP8: allocates the codes and scales (with torch,
on the weights' device) and calls mok_block_quantize, mok_block_quantize_weights, mok_block_gemm and
mok_block_wgrad. Argument marshalling only."""
from __future__ import annotations

import torch

from . import (_up128, block_padded_rows, mok_block_gemm, mok_block_quantize, mok_block_quantize_weights,
               mok_block_wgrad)


def _shape(t, name: str, *shape: int):
    if t.shape != shape:
        raise ValueError(f"{name} must be {shape}, not {tuple(t.shape)}")


class MokBlockLinear:
    """y[r] = x[r] w[g]^T for the rows r of every group (expert) g, weights w [G][N][K] float32 or bfloat16 kept by
    the caller. Rows [rows] are sorted by group, offsets int32 [G + 1] on the device as in a schedule table. With
    train, forward also keeps x's columns for the weight gradient, and the weights' transposes are made."""

    def __init__(self, w, rows: int, train: bool = True):
        self.w, self.rows, self.train = w, rows, train
        G, N, K = w.shape
        u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=w.device)
        f32 = lambda *s: torch.empty(s, dtype=torch.float32, device=w.device)
        P = block_padded_rows(rows, G)
        kb, nb, pb = _up128(K) // 128, _up128(N) // 128, P // 128
        self.wq, self.ws = u8(G, N, kb * 128), f32(G, nb, kb)
        self.xq, self.xs = u8(rows, kb * 128), f32(kb, rows)
        self.wt = self.wts = self.xt = self.xts = None
        if train:
            self.wt, self.wts = u8(G, K, nb * 128), f32(G, kb, nb)
            self.xt, self.xts = u8(K, P), f32(pb, K)
            self.yq, self.ys = u8(rows, nb * 128), f32(nb, rows)
            self.yt, self.yts = u8(N, P), f32(pb, N)
        self.refresh_weights()

    def _check_rows(self, t, name: str, columns: int, offsets):
        """Codes round widths up to 128, so the library's calls take some other widths for these."""
        _shape(t, name, self.rows, columns)
        if offsets is not None:
            _shape(offsets, "offsets", self.w.shape[0] + 1)
        elif self.w.shape[0] > 1:
            raise ValueError(f"offsets of {self.w.shape[0]} groups are needed")

    def refresh_weights(self):
        """After an update of w in place (an optimizer step): quantises it again."""
        mok_block_quantize_weights(self.w, self.wq, self.ws, codes_t=self.wt, scales_t=self.wts)

    def forward(self, x, out, offsets=None):
        """out [rows][N] = x [rows][K] w^T (each float32 or bfloat16); rows in no group are left as they are."""
        self._check_rows(x, "x", self.w.shape[2], offsets)
        _shape(out, "out", self.rows, self.w.shape[1])
        mok_block_quantize(x, self.xq, self.xs, codes_t=self.xt, scales_t=self.xts, offsets=offsets)
        mok_block_gemm(self.xq, self.xs, self.wq, self.ws, out, offsets=offsets)

    def backward(self, dy, dx=None, dw=None, offsets=None, accumulate: bool = False):
        """Of the last forward, with its offsets: dx [rows][K] = dy w (None: not wanted; rows in no group are left as they are) and dw
        [G][N][K] float32 = dy^T x (None: not wanted), or added to."""
        if not self.train:
            raise RuntimeError("the map was made without train")
        self._check_rows(dy, "dy", self.w.shape[1], offsets)
        if dx is not None:
            _shape(dx, "dx", self.rows, self.w.shape[2])
        if dw is not None:
            _shape(dw, "dw", *self.w.shape)
        cols = (self.yt, self.yts) if dw is not None else (None, None)
        rows = (self.yq, self.ys) if dx is not None else (None, None)
        if dx is None and dw is None:
            return
        mok_block_quantize(dy, *rows, codes_t=cols[0], scales_t=cols[1], offsets=offsets)
        if dx is not None:
            mok_block_gemm(self.yq, self.ys, self.wt, self.wts, dx, offsets=offsets)
        if dw is not None:
            mok_block_wgrad(self.yt, self.yts, self.xt, self.xts, dw, offsets=offsets, accumulate=accumulate,
                            rows=self.rows)
