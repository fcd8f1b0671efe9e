"""Oracle of the expert products (test infrastructure only).

Tokens sorted by expert: expert e has rows offsets[e] .. offsets[e + 1] of x
(tokens x k), y and dy (tokens x n), and weights w[e] (n x k).  float64 numpy,
one expert at a time, from y[t] = w[e] x[t] and its derivatives.
"""
from __future__ import annotations

import numpy as np


def spans(offsets, tokens):
    """(expert, first row, one past the last) of every expert; offsets are
    clamped to 0..tokens and to the largest one before them."""
    lo = min(max(int(offsets[0]), 0), tokens)
    out = []
    for e in range(len(offsets) - 1):
        hi = max(lo, min(max(int(offsets[e + 1]), 0), tokens))
        out.append((e, lo, hi))
        lo = hi
    return out


def expert_matmul(x, w, offsets, out):
    """out with y[t] in every expert's rows and the other rows as they were."""
    y = np.array(out, dtype=np.float64)
    for e, lo, hi in spans(offsets, len(x)):
        y[lo:hi] = x[lo:hi] @ w[e].T
    return y


def expert_input_grad(dy, w, offsets, out):
    dx = np.array(out, dtype=np.float64)
    for e, lo, hi in spans(offsets, len(dy)):
        dx[lo:hi] = dy[lo:hi] @ w[e]
    return dx


def expert_weight_grad(dy, x, offsets, out=None):
    """dw, added to ``out`` when given."""
    n_exp = len(offsets) - 1
    dw = np.zeros((n_exp, dy.shape[1], x.shape[1])) if out is None else np.array(out, dtype=np.float64)
    for e, lo, hi in spans(offsets, len(x)):
        dw[e] += dy[lo:hi].T @ x[lo:hi]
    return dw
