"""The large-tile and few-rows kernels with rows that have a stride, NaN in
every gap between rows and between experts, non-finite values in one
neighbouring expert and in rows of no expert; results in padded buffers.

Tolerances.  Expert products: sums of `length` products, exact in fp32, each
addition rounded once: (length + 2) 2^-24 S with S the sum of the magnitudes,
and half a bf16 step of the result.  8-bit products with bf16 results: the
matrix instruction adds eight consecutive products cut toward zero at 2^-13 of
the power of two of the largest one (the exponents' sum, so a subnormal or
zero operand counts as the format's smallest normal number): at most
8 * 2^-13 of it; the k / 8 sums join in fp32 (2^-23 of S each allowed), are
scaled (two roundings per block) and rounded to bf16 once."""
import pytest
import torch

from oracle import experts as oe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
Q8 = {"e4m3": (torch.float8_e4m3fn, -6), "e5m2": (torch.float8_e5m2, -14)}


def padded(gen, shape, std, before, after, dtype=BF):
    """Random values with `before` and `after` more rows and columns of NaN around
    each matrix; a view of the values."""
    full = list(shape)
    full[-1] += before[-1] + after[-1]
    if len(shape) == 3:
        full[-2] += before[0] + after[0]
    buf = torch.full(full, float("nan"), dtype=dtype, device=DEV)
    view = buf[..., before[-1]:before[-1] + shape[-1]]
    if len(shape) == 3:
        view = view[:, before[0]:before[0] + shape[-2]]
    view.copy_((torch.randn(shape, generator=gen, device=DEV) * std).to(dtype))
    return view


class Out:
    """A result inside a buffer of sevens."""

    def __init__(self, shape, dtype, rows=0, old=None):
        full = list(shape)
        full[-1] += 24
        if len(shape) == 3:
            full[-2] += rows
        self.buf = torch.full(full, 7.0, dtype=dtype, device=DEV)
        self.view = self.buf[..., 8:8 + shape[-1]]
        if len(shape) == 3:
            self.view = self.view[:, :shape[-2]]
        if old is not None:
            self.view.copy_(old)

    def gaps_are_untouched(self):
        got = self.view.clone()
        self.view.fill_(7.0)
        assert bool((self.buf == 7).all())
        return got


def within(got, ref, mag, length, out, what):
    tol = (length + 2) * 2.0 ** -24 * mag
    if out == BF:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    err = (got.double() - ref).abs()
    assert bool((err <= tol + 1e-37).all()), (what, float((err / (tol + 1e-37)).nan_to_num(9e9).max()))


# tokens, n, k, offsets (expert 2 holds the non-finite values); forward, input
# and weight gradient in 256 x 256 tiles (at least 128 by any offsets), then the
# forms of the few-rows kernel: 1 x 1 blocks of 16 with 16 and with 8 waves, 1 x 2, 2 x 2
LARGE_N = (720, 8200, 200, [5, 305, 305, 405, 605, 669])
LARGE_K = (720, 136, 8264, [5, 305, 305, 405, 605, 669])
FEW = [(33, 260, 520, [1, 1, 4, 20, 22, 31]), (33, 600, 520, [1, 4, 7, 20, 22, 31]),
       (33, 1800, 136, [0, 3, 3, 19, 21, 32]), (100, 72, 1032, [2, 41, 42, 72, 99])]


def bf16_case(lib, tokens, n, k, off, which):
    gen = torch.Generator(device=DEV).manual_seed(tokens + n)
    experts = len(off) - 1
    x = padded(gen, (tokens, k), 1.0, (8,), (16,))
    dy = padded(gen, (tokens, n), 0.1, (16,), (24,))
    w = padded(gen, (experts, n, k), 0.05, (3, 8), (5, 8))
    spans = oe.spans(off, tokens)
    inside = torch.zeros(tokens, dtype=torch.bool, device=DEV)
    for _, lo, hi in spans:
        inside[lo:hi] = True
    bad = spans[2]
    x[~inside], dy[~inside] = float("nan"), float("inf")
    x[bad[1]:bad[2]], dy[bad[1]:bad[2]], w[2] = float("nan"), float("nan"), float("inf")
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    X, W, DY = x.double(), w.double(), dy.double()
    if "f" in which or "d" in which:
        keep = torch.randn(tokens, n, generator=gen, device=DEV).to(BF)
        keep_x = torch.randn(tokens, k, generator=gen, device=DEV).to(BF)
        y, dx = Out((tokens, n), BF, old=keep), Out((tokens, k), BF, old=keep_x)
        lib.dmuon_expert_matmul(x, w, offs, out=y.view)
        lib.dmuon_expert_input_grad(dy, w, offs, out=dx.view)
        y, dx = y.gaps_are_untouched(), dx.gaps_are_untouched()
        assert torch.equal(y[~inside], keep[~inside]) and torch.equal(dx[~inside], keep_x[~inside])
        for e, lo, hi in spans:
            if e == 2:
                assert hi > lo and not bool(torch.isfinite(y[lo:hi]).any()) and not bool(torch.isfinite(dx[lo:hi]).any())
            elif hi > lo:
                t = W[e].t().contiguous()
                within(y[lo:hi], X[lo:hi] @ t, X[lo:hi].abs() @ t.abs(), k, BF, ("forward", e))
                within(dx[lo:hi], DY[lo:hi] @ W[e], DY[lo:hi].abs() @ W[e].abs(), n, BF, ("input", e))
    if "w" in which:
        for out in (BF, F32):
            for accumulate in (False, True):
                old = torch.randn(experts, n, k, generator=gen, device=DEV).to(out)
                dw = Out((experts, n, k), out, rows=3, old=old)
                lib.dmuon_expert_weight_grad(dy, x, offs, out=dw.view, accumulate=accumulate)
                dw = dw.gaps_are_untouched()
                for e, lo, hi in spans:
                    if e == 2:
                        assert not bool(torch.isfinite(dw[e]).any())
                        continue
                    t = DY[lo:hi].t().contiguous()
                    ref, mag = t @ X[lo:hi], t.abs() @ X[lo:hi].abs()
                    if accumulate:
                        ref, mag = ref + old[e].double(), mag + old[e].double().abs()
                    within(dw[e], ref, mag, hi - lo + 1, out, ("weight", e, accumulate))


@pytest.mark.parametrize("case", [LARGE_N, LARGE_K], ids=["wide-n", "wide-k"])
def test_large_tiles_bf16(lib, case):
    bf16_case(lib, *case, "fdw")


@pytest.mark.parametrize("case", FEW, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}")
def test_few_rows_bf16(lib, case):
    bf16_case(lib, *case, "f")


def quantised(gen, shape, block_rows, fmt, pad):
    """8-bit values as quantisation leaves them, NaN (0x7f) in the gaps, and scales."""
    dt, _ = Q8[fmt]
    full = shape[:-1] + (shape[-1] + pad,)
    buf = torch.full(full, 0x7f, dtype=torch.uint8, device=DEV)
    q = buf.view(dt)[..., 16:16 + shape[-1]]
    vals = (torch.randn(shape, generator=gen, device=DEV) * 100).clamp(-448, 448).to(dt)
    buf[..., 16:16 + shape[-1]] = vals.view(torch.uint8)
    rows = -(-shape[-2] // block_rows)
    s = torch.exp(torch.randn(shape[:-2] + (rows, -(-shape[-1] // 128)), generator=gen, device=DEV)) * 1e-3
    return q, s.float()


def values(q, s, block_rows, fmt):
    """(values, their powers of two) in float64, of one matrix."""
    rows, cols = q.shape
    at = torch.arange(rows, device=DEV) // block_rows
    sc = s.double()[at][:, torch.arange(cols, device=DEV) // 128]
    v = q.double()
    power = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** Q8[fmt][1]))))
    return v * sc, power * sc


def block_bound(a, pa, b, pb):
    """(reference, tolerance) of c = a @ b.T with bf16 results."""
    k = a.shape[1]
    bt = b.t().contiguous()
    ref, mag = a @ bt, a.abs() @ bt.abs()
    cut = torch.zeros_like(ref)
    for k0 in range(0, k, 8):
        top = torch.zeros_like(ref)
        for j in range(k0, min(k, k0 + 8)):
            top = torch.maximum(top, torch.outer(pa[:, j], pb[:, j]))
        cut += 8 * 2.0 ** -13 * top
    tol = cut + (2 * -(-k // 8) + 3 * -(-k // 128) + 3) * 2.0 ** -24 * mag
    return ref, tol + 2.0 ** -8 * (ref.abs() + tol) + 1e-37


# 256 x 256 tiles (at least 192 by any offsets) with an even and an odd number
# of blocks of k, one that ends inside a block; then the few-rows forms
@pytest.mark.parametrize("br", [128, 1])
@pytest.mark.parametrize("fmts", ["e4m3-e4m3", "e5m2-e4m3"])
@pytest.mark.parametrize("case", [(600, 8200, 400, [7, 7, 300, 340, 440, 590]), (610, 8200, 272, [3, 260, 300, 580, 610])]
                         + FEW, ids=lambda c: f"{c[0]}x{c[1]}x{c[2]}")
def test_block_product(lib, case, fmts, br):
    m, n, k, off = case
    k = k // 16 * 16
    fa, fb = fmts.split("-")
    gen = torch.Generator(device=DEV).manual_seed(m + n + br)
    experts = len(off) - 1
    a, sa = quantised(gen, (m, k), 1, fa, 48)
    b, sb = quantised(gen, (experts, n, k), br, fb, 64)
    spans = oe.spans(off, m)
    inside = torch.zeros(m, dtype=torch.bool, device=DEV)
    for _, lo, hi in spans:
        inside[lo:hi] = True
    bad = spans[2]
    a.view(torch.uint8)[~inside] = 0x7f
    sa[~inside] = float("inf")
    a.view(torch.uint8)[bad[1]:bad[2]] = 0x7f
    b.view(torch.uint8)[2] = 0x7f
    sa[bad[1]:bad[2]], sb[2] = float("nan"), float("inf")
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    keep = torch.randn(m, n, generator=gen, device=DEV).to(BF)
    out = Out((m, n), BF, old=keep)
    lib.dmuon_block_matmul(a, sa, b, sb, block_rows=br, offsets=offs, out=out.view)
    got = out.gaps_are_untouched()
    assert torch.equal(got[~inside], keep[~inside])
    full = Out((m, n), F32, old=keep)
    lib.dmuon_block_matmul(a, sa, b, sb, block_rows=br, offsets=offs, out=full.view)
    wide = full.gaps_are_untouched()
    assert torch.equal(wide[~inside], keep[~inside].float())
    for e, lo, hi in spans:
        if e == 2:
            assert hi > lo and not bool(torch.isfinite(got[lo:hi]).any()) and not bool(torch.isfinite(wide[lo:hi]).any())
        elif hi > lo:
            A, pa = values(a[lo:hi], sa[lo:hi], 1, fa)
            B, pb = values(b[e], sb[e], br, fb)
            ref, tol = block_bound(A, pa, B, pb)
            err = (got[lo:hi].double() - ref).abs()
            assert bool((err <= tol).all()), (e, float((err / tol).max()))
            within(wide[lo:hi], ref, A.abs() @ B.abs().t().contiguous(), k + 3 * -(-k // 128) + 1, F32, ("fp32", e))


@pytest.mark.parametrize("fmts", ["e4m3-e4m3", "e5m2-e4m3", "e4m3-e5m2", "e5m2-e5m2"])
@pytest.mark.parametrize("m,n", [(7, 64), (40, 72), (300, 130), (2000, 2100), (768, 16400)])
def test_sums_that_cancel(lib, m, n, fmts):
    """Each row of a holds pairs of opposite values against equal ones of b, the
    largest of the format among them, and a small remainder: the results are far
    smaller than the products.  Few-rows, 64-, 128- and 256-tiles."""
    fa, fb = fmts.split("-")
    gen = torch.Generator(device=DEV).manual_seed(m)
    k = 256
    av, bv = torch.randn(m, k, generator=gen, device=DEV) * 20, torch.randn(n, k, generator=gen, device=DEV) * 20
    for c in (0, 128):
        av[:, c], bv[:, c] = 448.0, 448.0          # an outlier column
        av[:, c + 60:c + 120], bv[:, c + 60:c + 120] = -av[:, c:c + 60], bv[:, c:c + 60]
    a, b = av.clamp(-448, 448).to(Q8[fa][0]), bv.clamp(-448, 448).to(Q8[fb][0])
    sa = torch.full((m, 2), 2.0 ** -5, device=DEV)
    sb = torch.full((n, 2), 2.0 ** -7, device=DEV)
    got = lib.dmuon_block_matmul(a, sa, b, sb, block_rows=1)
    A, pa = values(a, sa, 1, fa)
    B, pb = values(b, sb, 1, fb)
    ref, tol = block_bound(A, pa, B, pb)
    err = (got.double() - ref).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    wide = lib.dmuon_block_matmul(a, sa, b, sb, block_rows=1, out_dtype=F32)
    within(wide, ref, A.abs() @ B.abs().t().contiguous(), k + 9, F32, "fp32")


def test_what_the_instruction_keeps(lib):
    """Beside two products of 2^15 that cancel, a product of 2^2 (2^-13 of them) in
    the same eight is kept; in another eight one of 2^-7 is."""
    a = torch.zeros(4, 128, device=DEV)
    a[:, 0], a[:, 1] = 2.0 ** 15, -2.0 ** 15
    a[0, 2], a[1, 7], a[2, 8], a[3, 100] = 4.0, -4.0, 2.0 ** -7, -2.0 ** -7
    b = torch.ones(16, 128, device=DEV).to(torch.float8_e4m3fn)
    one = torch.ones(4, 1, device=DEV)
    c = lib.dmuon_block_matmul(a.to(torch.float8_e5m2), one, b, torch.ones(16, 1, device=DEV), block_rows=1)
    want = torch.tensor([4.0, -4.0, 2.0 ** -7, -2.0 ** -7], device=DEV).to(BF)
    assert torch.equal(c, want[:, None].expand(4, 16))
