"""Oracle of the 8-bit integer rows, their product and the expert layer, in numpy.

TEST INFRASTRUCTURE ONLY.  Quantisation is repeated in fp32, operation by
operation; sums and the layer are formed in float64 (int64 for integers).
"""
from __future__ import annotations

import numpy as np

F = np.float32


def quantize(x):
    """(q, scale) of fp32 rows."""
    x = np.asarray(x, F)
    scale = np.maximum(np.abs(x).max(-1) * (F(1) / F(127)), F(2.0 ** -126))
    return np.rint(x * (F(1) / scale)[..., None]).astype(np.int8), scale


def silu(a):
    with np.errstate(over="ignore"):
        return a / (1 + np.exp(-a))


def swiglu(x):
    x = np.asarray(x, np.float64)
    n = x.shape[-1] // 2
    return silu(x[..., :n]) * x[..., n:]


def matmul(a, a_scale, b, b_scale, offsets=None, c=None):
    """a (m x k) times b's rows, scaled; rows of no expert as in c."""
    a, sa, sb = a.astype(np.int64), a_scale.astype(np.float64), b_scale.astype(np.float64)
    if offsets is None:
        return (a @ b.astype(np.int64).T) * sa[:, None] * sb
    out = np.array(c, np.float64)
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        out[lo:hi] = (a[lo:hi] @ b[e].astype(np.int64).T) * sa[lo:hi, None] * sb[e]
    return out


def layer(x, ids, gates, w_in, w_out):
    """(y, the fp32 error's and the rounding's bound without y's own rounding) of a layer of
    experts; float64 weights.  A sum of len products in fp32 is off by (len + 8) 2^-24 of
    the sum of their magnitudes (operands, products, scale); silu in fp32 by
    (2 |a| + 16) 2^-23 of itself, and moves by at most 1.1 of its argument's error; h is held as two
    bf16 values, each off by half a step: 2^-16 of it."""
    tokens, top_k = ids.shape
    n, k = w_out.shape[2], w_out.shape[1]
    y, err, mag = np.zeros((tokens, k)), np.zeros((tokens, k)), np.zeros((tokens, k))
    u = 2.0 ** -24
    for t in range(tokens):
        for e in sorted(set(int(i) for i in ids[t] if 0 <= i < w_in.shape[0])):
            gate = gates[t][ids[t] == e].sum()
            a, b = w_in[e][:n] @ x[t], w_in[e][n:] @ x[t]
            da, db = ((k + 8) * u * (np.abs(w) @ np.abs(x[t])) for w in (w_in[e][:n], w_in[e][n:]))
            h = gate * silu(a) * b
            dh = np.abs(gate) * (1.1 * da * (np.abs(b) + db) + np.abs(silu(a)) * db) + np.abs(h) * (2 * np.abs(a) + 16) * 2 * u
            dh += 2.0 ** -16 * (np.abs(h) + dh) + 2.0 ** -133
            y[t] += w_out[e] @ h
            err[t] += np.abs(w_out[e]) @ dh
            mag[t] += np.abs(w_out[e]) @ (np.abs(h) + dh)
    return y, err + (2 * n * top_k + 8) * u * mag
