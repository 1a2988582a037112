"""Expert routing with scores, a balancing bias, groups, top-k and renormalised weights, and its
gradient, token by token in fp64.

For a token with logits x: scores s = sigmoid(x) or softmax(x); keys s + b (x without a bias); of the
groups of consecutive experts the best few stay, scored by their largest key or by the sum of their two
largest s + b; the top_k largest keys are chosen, ties to the lower id; the weights come from the scores
alone. An expert is able when its logit and its key are above -inf (NaN is not).
"""
from __future__ import annotations

import dataclasses
import math

import numpy as np


@dataclasses.dataclass(frozen=True)
class Gate:
    E: int
    K: int
    score: str = "softmax"        # or "sigmoid"
    groups: int = 1
    top_groups: int = 1
    group_score: str = "max"      # or "top2"
    renorm: bool = True
    scale: float = 1.0


def scores(gate: Gate, x: np.ndarray) -> np.ndarray:
    """s of one row; rows whose logits are all -inf have the score 0 everywhere."""
    x = np.asarray(x, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if gate.score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-x))
        top = np.max(x)
        if top == -math.inf:
            return np.zeros_like(x)
        z = np.exp(x - top)
        return z / z.sum()


def choose_row(gate: Gate, x, bias=None) -> list:
    """The chosen experts of one token, best first."""
    x = np.asarray(x, np.float64)
    s = scores(gate, x)
    b = None if bias is None else np.asarray(bias, np.float64)
    biased = s if b is None else s + b
    key = x if b is None else biased
    scored = b is not None or (gate.groups > 1 and gate.group_score == "top2")
    able = [e for e in range(gate.E)
            if x[e] > -math.inf and key[e] > -math.inf and (not scored or biased[e] > -math.inf)]
    if gate.groups > 1:
        size = gate.E // gate.groups
        value = []
        for g in range(gate.groups):
            of = [e for e in able if e // size == g]
            if not of:
                value.append(-math.inf)
            elif gate.group_score == "max":
                value.append(max(key[e] for e in of))
            else:
                value.append(sum(sorted((biased[e] for e in of), reverse=True)[:2]))
        kept = sorted(range(gate.groups), key=lambda g: (-value[g], g))[:gate.top_groups]
        able = [e for e in able if e // size in kept]
    return sorted(able, key=lambda e: (-key[e], e))[:gate.K]


def forward(gate: Gate, x, bias=None, mask=None):
    """(idx int32 [N][K], w fp64 [N][K], load int64 [E])"""
    x = np.asarray(x, np.float64)
    N = len(x)
    idx = np.full((N, gate.K), -1, np.int32)
    w = np.zeros((N, gate.K))
    load = np.zeros(gate.E, np.int64)
    for n in range(N):
        if mask is not None and not mask[n]:
            continue
        of = choose_row(gate, x[n], bias)
        idx[n, :len(of)] = of
        load[of] += 1
        w[n, :len(of)] = weights_row(gate, x[n], of)
    return idx, w, load


def weights_row(gate: Gate, x, of) -> np.ndarray:
    """Weights of the chosen experts `of` of one token. The quotient of scores is formed from the
    scores' logarithms less their largest, so it does not depend on the scores' size."""
    x = np.asarray(x, np.float64)
    if len(of) == 0:
        return np.zeros(0)
    if not gate.renorm:
        return gate.scale * scores(gate, x)[of]
    f = x[of] if gate.score == "softmax" else -np.logaddexp(0.0, -x[of])
    q = np.exp(f - f.max())
    return gate.scale * q / q.sum()


def backward(gate: Gate, x, idx, dw) -> np.ndarray:
    """dlogits fp64 [N][E] by the chain rule through the scores (sigmoid' = s (1 - s); softmax' =
    diag(s) - s s^T) and the quotient. dw at slots without an expert is not used."""
    x = np.asarray(x, np.float64)
    out = np.zeros(x.shape)
    for n in range(len(x)):
        slots = [k for k in range(gate.K) if idx[n, k] >= 0]
        if not slots:
            continue
        of = [int(idx[n, k]) for k in slots]
        g = np.asarray([dw[n, k] for k in slots], np.float64) * gate.scale
        if gate.renorm:
            # w = scale q, q = softmax(f); f' = 1, or sigmoid(-x)
            q = weights_row(dataclasses.replace(gate, scale=1.0), x[n], of)
            d = q * (g - (g * q).sum())
            if gate.score == "sigmoid":
                d = d * np.exp(-np.logaddexp(0.0, x[n][of]))
            out[n, of] = d
        elif gate.score == "sigmoid":
            out[n, of] = g * np.exp(-np.logaddexp(0.0, -x[n][of]) - np.logaddexp(0.0, x[n][of]))
        else:
            s = scores(gate, x[n])
            ds = np.zeros(gate.E)
            ds[of] = g
            out[n] = s * (ds - (s * ds).sum())
    return out
