"""8-bit block operators against the oracle.

Quantisation and its inverse are defined operation by operation in fp32, so
their results are compared bit for bit (fp32) or to one rounding (bf16).

Tolerances of the product.  fp32 results: operands are exact in bf16, a
block's sum is formed in fp32, multiplied by the rounded product of two
scales and added in fp32: with S the sum of the scaled products' magnitudes,
|got - ref| <= (k + 3 blocks + 3) 2^-24 S.  bf16 results: the 8-bit matrix
instruction keeps every product to at least 13 bits below the largest of its
128, so a block is off by at most 128 2^-13 of its largest scaled product, and
the result is rounded once (2^-8).  That bound is loose for sums of random
signs, so the whole result is also held to 2^-8 + 2^-10 in the Frobenius norm
(2^-8 is the rounding's largest share; 128 errors of 2^-13 at random add up to
sqrt(128) 2^-13 = 2^-9.5 of one product against a sum of 128).
"""
import numpy as np
import pytest
import torch

from oracle import blocks as ob
from oracle import experts as oe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
DT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def make(rng, shape, dtype, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype).to(DEV)


def host(t):
    return t.detach().float().cpu().numpy()


SHAPES = [(1, 1), (1, 128), (3, 129), (128, 128), (127, 384), (130, 100), (257, 300), (64, 1000), (300, 16), (5, 777)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize(lib, block_rows, fmt, dtype):
    rng = np.random.default_rng(block_rows)
    for rows, cols in SHAPES:
        x = make(rng, (rows, cols), dtype)
        x[:, ::37] *= 100
        x[rows // 2] *= 1e-20
        q, s, qt, st = lib.dmuon_quantize_blocks(x, block_rows=block_rows, fmt=fmt, transposed=True)
        for mat, got, scale in ((host(x), q, s), (host(x).T, qt, st)):
            want, ws = ob.quantize(mat, block_rows, fmt)
            assert np.array_equal(host(scale), ws), (rows, cols)
            assert np.array_equal(host(got).astype(np.float64), want), (rows, cols)
        only = lib.dmuon_quantize_blocks(x, block_rows=block_rows, fmt=fmt)
        assert torch.equal(only[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(only[1], s)
        assert only[2] is None and only[3] is None
        back = lib.dmuon_dequantize_blocks(q, s, block_rows=block_rows, dtype=dtype)
        ref = torch.from_numpy((host(q) * ob.spread(host(s), block_rows, rows, cols)).astype(np.float32)).to(dtype)
        assert torch.equal(back.cpu(), ref), (rows, cols)


def test_quantize_strides_and_batch(lib):
    rng = np.random.default_rng(11)
    for dtype in (BF, F32):
        big = make(rng, (3, 140, 420), dtype)
        for x in (big[:, 2:, 8:300], big[:, :133, 3:262], big[1:2, :, :256], big[0, :, 5:10]):
            for br in (1, 128):
                q, s, qt, st = lib.dmuon_quantize_blocks(x, block_rows=br, transposed=True)
                mats = [x] if x.dim() == 2 else list(x)
                for i, m in enumerate(mats):
                    pick = (lambda t: t) if x.dim() == 2 else (lambda t: t[i])
                    for mat, got, scale in ((host(m), q, s), (host(m).T, qt, st)):
                        want, ws = ob.quantize(mat, br, "e4m3")
                        assert np.array_equal(host(pick(scale)), ws)
                        assert np.array_equal(host(pick(got)).astype(np.float64), want)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_special_values(lib, block_rows):
    """Zeros, subnormals, the largest values, NaN and Inf: a non-finite value
    reaches its own block only."""
    x = torch.randn(256, 384, device=DEV)
    x[0, :128] = 0
    x[1, :128] = 1e-42
    x[2, :128] = 3e38
    x[130, 200] = float("nan")
    x[131, 300] = float("-inf")
    q, s, qt, st = lib.dmuon_quantize_blocks(x, block_rows=block_rows, transposed=True)
    back = lib.dmuon_dequantize_blocks(q, s, block_rows=block_rows, dtype=F32)
    r = (slice(130, 131), slice(131, 132)) if block_rows == 1 else (slice(128, 256), slice(128, 256))
    want = torch.zeros(256, 384, dtype=torch.bool)
    want[r[0], 128:256] = True
    want[r[1], 256:384] = True
    assert torch.equal(torch.isnan(back).cpu(), want)
    assert torch.equal(torch.isfinite(back).cpu(), ~want)
    back_t = lib.dmuon_dequantize_blocks(qt, st, block_rows=block_rows, dtype=F32).T
    want = torch.zeros(256, 384, dtype=torch.bool)
    want[128:256, slice(200, 201) if block_rows == 1 else slice(128, 256)] = True
    want[128:256, slice(300, 301) if block_rows == 1 else slice(256, 384)] = True
    assert torch.equal(torch.isnan(back_t).cpu(), want)


def quantized(rng, shape, block_rows, fmt):
    """8-bit values and scales with magnitudes as quantisation leaves them."""
    rows, cols = shape[-2:]
    q = torch.from_numpy(np.clip(rng.standard_normal(shape) * 100, -448, 448).astype(np.float32)).to(DT[fmt]).to(DEV)
    s = np.exp(rng.standard_normal(shape[:-2] + (-(-rows // block_rows), -(-cols // 128)))) * 1e-3
    return q, torch.from_numpy(s.astype(np.float32)).to(DEV)


def check(got, a, sa, b, sb, br, old=None):
    """One product against the oracle, by the bounds of the module's header."""
    fp32 = got.dtype == F32
    got = got.double().cpu().numpy()
    A, B = ob.dequantize(host(a), host(sa), 1), ob.dequantize(host(b), host(sb), br)
    ref, S = A @ B.T, np.abs(A) @ np.abs(B).T
    k = A.shape[1]
    if old is not None:
        ref, S = ref + host(old), S + np.abs(host(old))
    if fp32:
        tol = (k + 3 * -(-k // 128) + 4) * 2.0 ** -24 * S + 1e-37
    else:
        tol = 2.0 ** -8 * np.abs(ref) + 1e-37
        for kb in range(0, k, 128):
            top = (np.abs(A[:, None, kb:kb + 128]) * np.abs(B[None, :, kb:kb + 128])).max(axis=2)
            tol = tol + 128 * 2.0 ** -13 * top
        fro = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert fro <= 2.0 ** -8 + 2.0 ** -10, fro
    bad = np.abs(got - ref) > tol * (1 + 1e-6)
    assert not bad.any(), (int(bad.sum()), float((np.abs(got - ref) / tol).max()))


PRODUCTS = [(1, 1, 1), (2, 40, 130), (7, 256, 512), (16, 100, 16), (33, 129, 257), (128, 128, 128), (130, 260, 384),
            (200, 72, 1000), (300, 300, 48), (5, 4200, 144), (20, 8200, 272), (16, 36, 2064)]


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("br", [128, 1])
@pytest.mark.parametrize("fmts", ["e4m3-e4m3", "e5m2-e4m3", "e4m3-e5m2", "e5m2-e5m2"])
def test_product(lib, fmts, br, out):
    rng = np.random.default_rng(13)
    fa, fb = fmts.split("-")
    for m, n, k in PRODUCTS:
        a, sa = quantized(rng, (m, k), 1, fa)
        b, sb = quantized(rng, (n, k), br, fb)
        got = lib.dmuon_block_matmul(a, sa, b, sb, block_rows=br, out_dtype=out)
        assert got.dtype == out
        check(got, a, sa, b, sb, br)
        old = make(rng, (m, n), out)
        acc = old.clone()
        lib.dmuon_block_matmul(a, sa, b, sb, block_rows=br, out=acc, accumulate=True)
        check(acc, a, sa, b, sb, br, old)


@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("br", [128, 1])
def test_expert_product(lib, br, out):
    rng = np.random.default_rng(14)
    for m, n, k, off in ((1, 16, 32, [0, 0, 1]), (9, 130, 272, [1, 1, 4, 8]), (300, 200, 400, [0, 128, 128, 300]),
                         (400, 64, 100, [10, 20, 390]), (64, 136, 256, list(range(65))),
                         (90, 30, 60, [-4, 70, 20, 999])):
        e = len(off) - 1
        a, sa = quantized(rng, (m, k), 1, "e4m3")
        b, sb = quantized(rng, (e, n, k), br, "e4m3")
        keep = make(rng, (m, n), out)
        got = keep.clone()
        offs = torch.tensor(off, dtype=torch.int32, device=DEV)
        lib.dmuon_block_matmul(a, sa, b, sb, block_rows=br, offsets=offs, out=got)
        outside = torch.ones(m, dtype=torch.bool)
        for i, lo, hi in oe.spans(off, m):
            if hi > lo:
                check(got[lo:hi], a[lo:hi], sa[lo:hi], b[i], sb[i], br)
                outside[lo:hi] = False
        assert torch.equal(got[outside.to(DEV)], keep[outside.to(DEV)])


def test_product_strides(lib):
    rng = np.random.default_rng(15)
    a, sa = quantized(rng, (50, 300), 1, "e4m3")
    b, sb = quantized(rng, (70, 300), 128, "e4m3")
    for pad, shift in ((20, 0), (84, 16), (31, 5)):
        A = torch.zeros(50, 300 + pad, dtype=a.dtype, device=DEV)
        B = torch.zeros(70, 300 + pad, dtype=a.dtype, device=DEV)
        A.view(torch.uint8).fill_(0x7f)      # NaN around the rows
        B.view(torch.uint8).fill_(0x7f)
        A[:, shift:shift + 300], B[:, shift:shift + 300] = a, b
        big = torch.full((50, 100), 3.0, dtype=BF, device=DEV)
        lib.dmuon_block_matmul(A[:, shift:shift + 300], sa, B[:, shift:shift + 300], sb, out=big[:, shift:shift + 70])
        check(big[:, shift:shift + 70], a, sa, b, sb, 128)
        big[:, shift:shift + 70] = 3
        assert (big == 3).all()


def test_replays(lib):
    rng = np.random.default_rng(16)
    x, w = make(rng, (200, 260), BF), make(rng, (3, 100, 260), BF, 0.05)
    offs = torch.tensor([0, 50, 50, 190], dtype=torch.int32, device=DEV)
    q, s, qt, st = lib.dmuon_quantize_blocks(x, transposed=True)
    wq, ws, _, _ = lib.dmuon_quantize_blocks(w, block_rows=128)
    y = torch.zeros(200, 100, dtype=BF, device=DEV)

    def go():
        lib.dmuon_quantize_blocks(x, q=q, scale=s, qt=qt, scale_t=st)
        lib.dmuon_quantize_blocks(w, block_rows=128, q=wq, scale=ws)
        lib.dmuon_block_matmul(q, s, wq, ws, offsets=offs, out=y)

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for new in ([0, 50, 50, 190], [0, 0, 150, 200], [3, 3, 3, 3]):
        offs.copy_(torch.tensor(new, dtype=torch.int32))
        x.mul_(-1.5)
        y.zero_()
        go()
        torch.cuda.synchronize()
        want = [t.clone() for t in (q, s, qt, st, wq, ws, y)]
        y.zero_()
        q.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip((q, s, qt, st, wq, ws, y), want):
            assert torch.equal(got.view(torch.uint8) if got.element_size() == 1 else got,
                               ref.view(torch.uint8) if ref.element_size() == 1 else ref), new


@pytest.mark.parametrize("br", [128, 1])
@pytest.mark.parametrize("fmts", ["e4m3-e4m3", "e5m2-e4m3"])
def test_product_large_tiles(lib, fmts, br):
    """Enough 256 x 256 tiles for the kernel of that size: whole and short row
    tiles, a last column tile, an odd and an even number of blocks, a sum that
    ends inside a block; one product and experts.  A block's largest product is
    bounded here by the product of the two rows' largest values."""
    rng = np.random.default_rng(17)
    fa, fb = fmts.split("-")

    def large_check(got, a, sa, b, sb, old=None):
        A, B = ob.dequantize(host(a), host(sa), 1), ob.dequantize(host(b), host(sb), br)
        ref = A @ B.T + (0 if old is None else host(old))
        got = got.double().cpu().numpy()
        tol = 2.0 ** -8 * np.abs(ref) + 1e-37
        for kb in range(0, A.shape[1], 128):
            tol = tol + 128 * 2.0 ** -13 * np.outer(np.abs(A[:, kb:kb + 128]).max(1), np.abs(B[:, kb:kb + 128]).max(1))
        assert np.all(np.abs(got - ref) <= tol * (1 + 1e-6))
        assert np.linalg.norm(got - ref) <= (2.0 ** -8 + 2.0 ** -10) * np.linalg.norm(ref)

    for m, n, k in ((700, 12300, 272), (300, 16400, 144), (356, 16384, 384)):
        a, sa = quantized(rng, (m, k), 1, fa)
        b, sb = quantized(rng, (n, k), br, fb)
        large_check(lib.dmuon_block_matmul(a, sa, b, sb, block_rows=br), a, sa, b, sb)
        old = make(rng, (m, n), BF)
        acc = old.clone()
        lib.dmuon_block_matmul(a, sa, b, sb, block_rows=br, out=acc, accumulate=True)
        large_check(acc, a, sa, b, sb, old)
    m, n, k, off = 600, 6200, 160, [7, 7, 300, 340, 440, 590]
    a, sa = quantized(rng, (m, k), 1, fa)
    b, sb = quantized(rng, (5, n, k), br, fb)
    keep = make(rng, (m, n), BF)
    got = keep.clone()
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    lib.dmuon_block_matmul(a, sa, b, sb, block_rows=br, offsets=offs, out=got)
    for i, lo, hi in oe.spans(off, m):
        if hi > lo:
            large_check(got[lo:hi], a[lo:hi], sa[lo:hi], b[i], sb[i])
    assert torch.equal(got[:7], keep[:7]) and torch.equal(got[590:], keep[590:])
