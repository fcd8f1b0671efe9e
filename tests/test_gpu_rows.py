"""8-bit integer rows and their product against the oracle.

Quantisation without an activation is fp32 operation by operation, so integers and
scales have to be equal.  Gated: silu(g) u in fp32 is off by (2 |g| + 16) 2^-23 of
itself, the scale by that of its row's largest, and a value by half a scale on
top.  Product: the sum is exact; its conversion and two products round by 2^-24
each, an old value's addition by one more, and the result by half a step of its
type (2^-8 for bf16)."""
import numpy as np
import pytest
import torch

from oracle import rows as orow

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    import matrix_optimizer_step_owned_amd as dm
    return dm


def real(rng, shape, dtype, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(DEV).to(dtype)


def ints(rng, shape):
    return torch.from_numpy(rng.integers(-128, 128, shape, dtype=np.int8)).to(DEV)


def scales(rng, shape):
    return torch.from_numpy(np.exp(rng.standard_normal(shape)).astype(np.float32) * 0.01).to(DEV)


def host(t):
    return t.float().cpu().numpy()


ROWS = [(1, 1), (3, 7), (5, 8), (2, 9), (7, 511), (4, 512), (3, 513), (1025, 515), (1030, 2040), (1024, 4096),
        (1027, 1025), (6, 4097), (3, 16384), (3, 16385), (2, 40003), (1100, 33)]


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize(lib, rows, cols, dtype):
    rng = np.random.default_rng(rows + cols)
    x = real(rng, (rows, cols + 3), dtype, 3.0)
    x[:, ::5] *= 1e-3
    for v in (x[:, :cols].contiguous(), x[:, 2:cols + 2]):        # dense, and strided rows at an odd address
        buf = torch.full((rows * cols + 40,), 55, dtype=torch.int8, device=DEV)
        q, s = buf[20:20 + rows * cols].view(rows, cols), torch.empty(rows, device=DEV)
        lib.dmuon_quantize_rows(v, q=q, scale=s)
        rq, rs = orow.quantize(host(v))
        assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)
        assert (buf[:20] == 55).all() and (buf[20 + rows * cols:] == 55).all()
    for out in (BF, F32):
        got = lib.dmuon_dequantize_rows(q, s, dtype=out)
        assert torch.equal(got, (q.float() * s[:, None]).to(out))
    wide = torch.full((rows, cols + 5), 9.0, device=DEV)
    lib.dmuon_dequantize_rows(q, s, out=wide[:, 1:cols + 1])
    assert torch.equal(wide[:, 1:cols + 1], q.float() * s[:, None])
    assert (wide[:, 0] == 9).all() and (wide[:, cols + 1:] == 9).all()


@pytest.mark.parametrize("rows,cols", ROWS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_quantize_gated(lib, rows, cols, dtype):
    rng = np.random.default_rng(rows * 3 + cols)
    x = real(rng, (rows, 2 * cols + 1), dtype, 4.0)[:, 1:]
    if cols > 8:
        x[0, :4] = torch.tensor([80.0, -80.0, 100.0, -120.0]).to(x)
    q, s = lib.dmuon_quantize_rows(x, activation="swiglu")
    h, g = orow.swiglu(host(x)), np.abs(host(x)[:, :cols].astype(np.float64))
    rel = (2 * g.max(1) + 16) * 2.0 ** -23 + 2.0 ** -22      # the scale's two roundings too
    want = np.maximum(np.abs(h).max(1) / 127, 2.0 ** -126)
    got_s = s.double().cpu().numpy()
    assert (np.abs(got_s - want) <= rel * want).all()
    got = q.double().cpu().numpy() * got_s[:, None]
    assert (np.abs(got - h) <= (0.5 + 127 * rel[:, None]) * got_s[:, None] * (1 + 1e-6)).all()


def test_quantize_special_rows(lib):
    """Zeros, subnormal rows, one value, NaN and Inf in their own rows only; ties to even."""
    x = torch.zeros(9, 600, device=DEV)
    x[1, 17] = -5.0
    x[2] = 1e-42
    x[3, 599] = float("nan")
    x[4, 0] = float("inf")
    x[5, :4] = torch.tensor([127.0, 0.5, 1.5, -2.5])
    x[6, 300] = -float("inf")
    x[7] = 3e38
    q, s = lib.dmuon_quantize_rows(x)
    rq, rs = orow.quantize(host(x)[[0, 1, 2, 5, 7, 8]])
    keep = [0, 1, 2, 5, 7, 8]
    assert np.array_equal(q.cpu().numpy()[keep], rq) and np.array_equal(s.cpu().numpy()[keep], rs)
    assert q[5, :4].tolist() == [127, 0, 2, -2]
    got = lib.dmuon_dequantize_rows(q, s, dtype=F32)
    for r in range(9):
        assert torch.isnan(got[r]).all() == (r in (3, 4, 6)), r
        assert torch.isfinite(got[r]).all() == (r not in (3, 4, 6)), r
    y = torch.zeros(3, 20, dtype=BF, device=DEV)
    y[0, 10:], y[0, 0], y[1, 3], y[2, :] = 1, -float("inf"), float("nan"), 1
    got = lib.dmuon_dequantize_rows(*lib.dmuon_quantize_rows(y, activation="swiglu"), dtype=F32)
    assert torch.isnan(got[:2]).all() and torch.isfinite(got[2]).all()


def test_quantize_batches(lib):
    """Weights of experts: any leading dimensions; empty ones."""
    rng = np.random.default_rng(2)
    w = real(rng, (3, 5, 48), BF)
    q, s = lib.dmuon_quantize_rows(w)
    rq, rs = orow.quantize(host(w))
    assert q.shape == w.shape and s.shape == (3, 5)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)
    assert torch.equal(lib.dmuon_dequantize_rows(q, s, dtype=F32), q.float() * s[..., None])
    q, s = lib.dmuon_quantize_rows(w[:, :0].contiguous())
    assert q.shape == (3, 0, 48) and s.shape == (3, 0)


# ---- product ------------------------------------------------------------------

def tolerance(ref, dtype, old=0.0):
    return (4 * 2.0 ** -24 * (np.abs(ref - old) + np.abs(old) + np.abs(ref))
            + (2.0 ** -8 if dtype == BF else 0) * np.abs(ref) + 1e-38)


def compare(got, ref, dtype, old=0.0, what=""):
    got = got.double().cpu().numpy()
    tol = tolerance(ref, dtype, old)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all(), (what, float((np.abs(got - ref) / tol).max()))


# few rows, 64- and 128-tiles, 256-tiles (whole, odd, short), one of each size
SIZES = [(1, 1, 1), (1, 16, 64), (3, 5, 17), (7, 200, 128), (16, 33, 144), (17, 130, 256), (32, 48, 1040), (33, 70, 90),
         (100, 129, 127), (130, 257, 272), (512, 1000, 515), (700, 900, 1024), (300, 8200, 400), (7, 9000, 2064),
         (3100, 4096, 656), (4096, 3333, 128), (513, 24600, 96)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_matmul(lib, m, n, k, dtype):
    rng = np.random.default_rng(m + n + k)
    a, b, sa, sb = ints(rng, (m, k)), ints(rng, (n, k)), scales(rng, m), scales(rng, n)
    ref = orow.matmul(*[t.cpu().numpy() for t in (a, sa, b, sb)]) if m * n * k < 1e9 else None
    if ref is None:      # float64 is exact here too: sums below 2^53
        ref = ((a.double() @ b.double().T.contiguous()) * sa.double()[:, None] * sb.double()).cpu().numpy()
    compare(lib.dmuon_row_matmul(a, sa, b, sb, out_dtype=dtype), ref, dtype)
    # strided rows, a strided result between guards, added to what is there
    wide_a, wide_b = ints(rng, (m, k + 16)), ints(rng, (n, k + 32))
    wide_a[:, :k], wide_b[:, 16:16 + k] = a, b
    c = real(rng, (m + 2, n + 8), dtype)
    before = c.clone()
    lib.dmuon_row_matmul(wide_a[:, :k], sa, wide_b[:, 16:16 + k], sb, out=c[1:m + 1, 4:n + 4], accumulate=True)
    old = before[1:m + 1, 4:n + 4].double().cpu().numpy()
    compare(c[1:m + 1, 4:n + 4], ref + old, dtype, old)
    inside = torch.zeros_like(c, dtype=torch.bool)
    inside[1:m + 1, 4:n + 4] = True
    assert torch.equal(c[~inside], before[~inside])


OFFSETS = [(5, 16, 32, [0, 0, 1, 1, 5]), (40, 70, 90, [2, 9, 9, 33]), (64, 130, 256, list(range(0, 65, 4))),
           (130, 129, 272, [0, 128, 129, 129, 130]), (333, 200, 144, [3, 300, 330]),
           (720, 8200, 208, [5, 305, 305, 405, 605, 669]), (1300, 4096, 1040, [0, 256, 956, 968, 1268]),
           (96, 2000, 512, [0, 30, 31, 60, 96])]


@pytest.mark.parametrize("m,n,k,off", OFFSETS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_matmul_experts(lib, m, n, k, off, dtype, accumulate):
    rng = np.random.default_rng(m + n)
    e = len(off) - 1
    a, sa, sb = ints(rng, (m, k)), scales(rng, m), scales(rng, (e, n))
    store = ints(rng, (e, n + 3, k))
    b = store[:, :n]                       # experts further apart than their weights
    c = real(rng, (m, n), dtype)
    old = c.double().cpu().numpy()
    lib.dmuon_row_matmul(a, sa, b, sb, offsets=torch.tensor(off, dtype=torch.int32, device=DEV), out=c,
                         accumulate=accumulate)
    ref = orow.matmul(*[t.cpu().numpy() for t in (a, sa, b, sb)], off, old)
    inside = np.zeros(m, bool)
    inside[off[0]:off[-1]] = True
    base = old if accumulate else 0 * old
    ref[inside] += base[inside]
    compare(c[torch.from_numpy(inside).to(DEV)], ref[inside], dtype, base[inside])
    assert np.array_equal(c.double().cpu().numpy()[~inside], old[~inside])
    fresh = lib.dmuon_row_matmul(a, sa, b, sb, offsets=torch.tensor(off, dtype=torch.int32, device=DEV), out_dtype=dtype)
    assert (fresh[torch.from_numpy(~inside).to(DEV)] == 0).all()


def test_matmul_largest_sums(lib):
    """k at the limit with the extreme operands: sums of 2^31 - 2^14."""
    k = 131071
    a = torch.full((20, k), -128, dtype=torch.int8, device=DEV)
    b = torch.full((40, k), -128, dtype=torch.int8, device=DEV)
    b[1] = 127
    one = lambda n: torch.ones(n, device=DEV)
    got = lib.dmuon_row_matmul(a, one(20), b, one(40), out_dtype=F32)
    want = np.full((20, 40), np.float32(16384 * k))
    want[:, 1] = np.float32(-128 * 127 * k)
    assert np.array_equal(got.cpu().numpy(), want)


def test_matmul_not_finite_scales_stay_in_their_row(lib):
    rng = np.random.default_rng(4)
    for m, n, k in ((10, 40, 64), (700, 900, 1024), (3100, 4096, 256)):
        a, b, sa, sb = ints(rng, (m, k)), ints(rng, (n, k)), scales(rng, m), scales(rng, n)
        sa[3], sb[5] = float("nan"), float("nan")
        got = torch.isnan(lib.dmuon_row_matmul(a, sa, b, sb))
        assert got[3].all() and got[:, 5].all()
        got[3] = got[:, 5] = False
        assert not got.any()


def test_matmul_bad_offsets_stay_inside(lib):
    """Offsets that break the rules are clamped: nothing outside c is written."""
    rng = np.random.default_rng(5)
    m, n, k, e = 300, 264, 64, 4
    a, sa, b, sb = ints(rng, (m, k)), scales(rng, m), ints(rng, (e, n, k)), scales(rng, (e, n))
    for off in ([-5, 100, 50, 400, 1000], [400, 0, 0, 0, 0], [0, -1, -1, -1, -1], [7, 7, 7, 7, 7]):
        buf = torch.full((m + 20, n), 3.0, device=DEV)
        lib.dmuon_row_matmul(a, sa, b, sb, offsets=torch.tensor(off, dtype=torch.int32, device=DEV), out=buf[10:-10])
        torch.cuda.synchronize()
        assert (buf[:10] == 3).all() and (buf[-10:] == 3).all()


def test_matmul_graph_and_streams(lib):
    """Replays after eager work, on a stream of its own; two calls at once."""
    rng = np.random.default_rng(6)
    shapes = [(5, 512, 1024), (300, 700, 520), (3100, 4096, 256)]
    ops = [(ints(rng, (m, k)), scales(rng, m), ints(rng, (n, k)), scales(rng, n)) for m, n, k in shapes]
    eager = [lib.dmuon_row_matmul(*o) for o in ops]
    outs = [torch.zeros_like(x) for x in eager]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            for o, c in zip(ops, outs):
                lib.dmuon_row_matmul(*o, out=c)
    for _ in range(3):
        for c in outs:
            c.zero_()
        torch.cuda.synchronize()
        graph.replay()
        again = [lib.dmuon_row_matmul(*o) for o in ops]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(eager, outs, again))


def test_matmul_far_operands(lib):
    """Offsets past 2^32 bytes in each operand."""
    rng = np.random.default_rng(7)
    k, pitch = 64, 1 << 26
    for m, n in ((70, 40), (3, 5)):
        store = torch.zeros(72 * pitch, dtype=torch.int8, device=DEV)
        a, b = ints(rng, (m, k)), ints(rng, (n, k))
        sa, sb = scales(rng, m), scales(rng, n)
        far_a, far_b = (store[o:].as_strided((r, k), (pitch, 1)) for o, r in ((0, m), (4096, n)))
        far_a.copy_(a)
        far_b.copy_(b)
        assert torch.equal(lib.dmuon_row_matmul(far_a, sa, far_b, sb), lib.dmuon_row_matmul(a, sa, b, sb))
        e = 2
        w = store[8192:].as_strided((e, n, k), (70 * pitch // 16 * 16, k, 1))
        w.copy_(torch.stack((b, -b.clamp_min(-127))))
        off = torch.tensor([0, m // 2, m], dtype=torch.int32, device=DEV)
        sbe = torch.stack((sb, sb))
        assert torch.equal(lib.dmuon_row_matmul(a, sa, w, sbe, offsets=off),
                           lib.dmuon_row_matmul(a, sa, w.contiguous(), sbe, offsets=off))
        del store
