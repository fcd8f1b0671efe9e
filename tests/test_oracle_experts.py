"""Pins of the oracles of the expert products and the 8-bit blocks (CPU)."""
import numpy as np
import pytest
import torch

from oracle import blocks as ob
from oracle import experts as oe


def test_products_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    w = np.array([[[1.0, 0.0]], [[0.0, 10.0]]])
    y = oe.expert_matmul(x, w, [0, 1, 3], np.full((3, 1), 7.0))
    assert y.tolist() == [[1.0], [40.0], [60.0]]
    # rows of no expert stay, an expert without rows uses none
    y = oe.expert_matmul(x, w, [1, 1, 2], np.full((3, 1), 7.0))
    assert y.tolist() == [[7.0], [40.0], [7.0]]
    dw = oe.expert_weight_grad(np.ones((3, 1)), x, [0, 0, 2], np.ones((2, 1, 2)))
    assert dw.tolist() == [[[1.0, 1.0]], [[5.0, 7.0]]]


def test_spans_of_broken_offsets():
    assert oe.spans([-5, 2, 1, 99], 4) == [(0, 0, 2), (1, 2, 2), (2, 2, 4)]


def test_gradients_against_differences():
    """The products are bilinear, so a central difference is exact up to rounding."""
    rng = np.random.default_rng(0)
    off = [1, 3, 3, 6]
    x, w = rng.standard_normal((7, 5)), rng.standard_normal((3, 4, 5))
    dy = rng.standard_normal((7, 4))

    def loss(x, w):
        return float((oe.expert_matmul(x, w, off, np.zeros((7, 4))) * dy).sum())

    dx = oe.expert_input_grad(dy, w, off, np.zeros((7, 5)))
    dw = oe.expert_weight_grad(dy, x, off)
    for arr, grad in ((x, dx), (w, dw)):
        for _ in range(20):
            i = tuple(rng.integers(0, s) for s in arr.shape)
            keep = arr[i]
            arr[i] = keep + 0.5
            hi = loss(x, w)
            arr[i] = keep - 0.5
            lo = loss(x, w)
            arr[i] = keep
            assert abs((hi - lo) - grad[i]) < 1e-12


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_grid_is_torchs(fmt):
    dt = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    codes = torch.arange(256, dtype=torch.uint8).view(dt).float()
    vals = np.unique(codes[torch.isfinite(codes)].double().numpy())
    assert vals.max() == ob.FORMATS[fmt]["top"]
    mid = (vals[1:] + vals[:-1]) / 2
    v = np.concatenate([vals, mid, np.random.default_rng(1).uniform(-448, 448, 4000),
                        np.random.default_rng(2).uniform(-2.0 ** -8, 2.0 ** -8, 4000)])
    v = v.astype(np.float32)
    assert np.array_equal(ob.round_to_grid(v.astype(np.float64), fmt), torch.from_numpy(v).to(dt).double().numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_keeps_the_largest_and_bounds_the_rest(fmt, block_rows):
    x = np.random.default_rng(3).standard_normal((150, 300)).astype(np.float32)
    x[:, 128:256] = 0
    q, s = ob.quantize(x, block_rows, fmt)
    assert s.shape == (-(-150 // block_rows), 3)
    assert np.all(s[:, 1] == ob.SCALE_MIN) and not q[:, 128:256].any()
    assert np.abs(q).max() == ob.FORMATS[fmt]["top"]
    back = ob.dequantize(q, s, block_rows)
    half = 2.0 ** -(ob.FORMATS[fmt]["bits"] + 1)
    low = np.ldexp(1.0, ob.FORMATS[fmt]["low"]) * half
    bound = half * np.abs(x) + low * ob.spread(s, block_rows, 150, 300)
    assert np.all(np.abs(back - x) <= bound * (1 + 1e-6))


def test_block_product_by_hand():
    a, b = np.ones((1, 256)), np.ones((1, 256))
    got = ob.block_matmul(a, np.array([[2.0, 3.0]]), b, np.array([[5.0, 7.0]]), 1)
    assert got.tolist() == [[128 * 10.0 + 128 * 21.0]]
