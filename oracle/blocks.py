"""Oracle of the 8-bit block operators (test infrastructure only).

quantize: scale = max(amax / M, 2^-126) of every block_rows x 128 block and
x * (1 / scale), each operation in IEEE float32 as the operator is defined,
then rounded to the 8-bit grid, ties to even.  dequantize and block_matmul in
float64.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
FORMATS = {"e4m3": dict(bits=3, low=-6, top=448.0), "e5m2": dict(bits=2, low=-14, top=57344.0)}
SCALE_MIN = np.float32(2.0 ** -126)


def round_to_grid(v, fmt):
    """float64 values rounded to the format's nearest value, ties to even."""
    f = FORMATS[fmt]
    with np.errstate(divide="ignore"):
        exp = np.maximum(np.floor(np.log2(np.abs(v))), f["low"])
    exp = np.where(np.isfinite(exp), exp, f["low"])
    step = np.ldexp(1.0, (exp - f["bits"]).astype(int))
    return np.rint(v / step) * step


def block_max(x, block_rows):
    rows, cols = x.shape
    out = np.zeros((-(-rows // block_rows), -(-cols // BLOCK)), x.dtype)
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            out[i, j] = np.abs(x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]).max()
    return out


def spread(scale, block_rows, rows, cols):
    return np.repeat(np.repeat(scale, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]


def quantize(x, block_rows, fmt):
    """(values on the grid, float32 scales) of a float32 matrix."""
    x = np.asarray(x, np.float32)
    scale = np.maximum(block_max(x, block_rows) / np.float32(FORMATS[fmt]["top"]), SCALE_MIN)
    inv = np.float32(1.0) / scale
    return round_to_grid((x * spread(inv, block_rows, *x.shape)).astype(np.float64), fmt), scale


def dequantize(q, scale, block_rows):
    return q.astype(np.float64) * spread(scale.astype(np.float64), block_rows, *q.shape)


def block_matmul(a, a_scale, b, b_scale, block_rows):
    return dequantize(a, a_scale, 1) @ dequantize(b, b_scale, block_rows).T
