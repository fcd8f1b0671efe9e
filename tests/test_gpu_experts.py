"""Expert products against the float64 oracle.

Tolerances.  A result is a sum of `len` products of values that are exact in
float64, formed in fp32 (each product exact or rounded once, each addition
rounded once) and rounded once to the result's type: with S the sum of the
products' magnitudes,
    |got - ref| <= (len + 2) 2^-24 S + half a step of the result's type,
2^-8 |ref| for bf16, 2^-24 |ref| for fp32 (covered by the first term's + 2).
With accumulate the old value joins the sum.
"""
import numpy as np
import pytest
import torch

from oracle import experts as oe

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def make(rng, shape, dtype, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).to(dtype).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def check(got, ref, mag, length, dtype, what=""):
    """Every value within the derived bound; values are finite."""
    got = f64(got)
    assert np.isfinite(got).all(), what
    tol = (length + 2) * 2.0 ** -24 * mag + (2.0 ** -8 * np.abs(ref) if dtype == BF else 0) + 1e-37
    bad = np.abs(got - ref) > tol * (1 + 1e-6)
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - ref) / tol).max()))


def offsets_of(counts, first=0):
    return [first] + [int(v) for v in first + np.cumsum(counts)]


# (tokens, n, k, offsets): sizes below, at and past the tiles; experts without
# rows at the start, in the middle and at the end; rows of no expert
CASES = [
    (1, 1, 1, [0, 1]),
    (5, 16, 8, [0, 0, 1, 1, 5]),
    (7, 40, 24, [2, 2, 3, 6]),
    (130, 129, 257, offsets_of([0, 128, 1, 0, 1])),
    (300, 128, 64, offsets_of([127, 0, 129, 30], 5)),
    (333, 200, 136, offsets_of([333])),
    (517, 264, 328, offsets_of([256, 1, 255, 0, 5])),
    (640, 515, 70, offsets_of([3] * 100)),
    (1000, 384, 512, offsets_of([600, 400])),
    (64, 1000, 777, offsets_of([1] * 64)),
    # few rows per expert: one and two blocks of 16 rows, 16, 8 and 4 waves
    (33, 260, 520, offsets_of([1, 0, 3, 16, 2, 11])),
    (100, 72, 1032, offsets_of([40, 1, 30, 29])),
    (9, 2100, 136, offsets_of([2, 6], 1)),
    (45, 8200, 72, offsets_of([2, 43])),
    # enough 256 x 256 tiles for the kernel of that size: row tiles of 256,
    # 200, 100 and 44 rows, a sum that ends inside a stage
    (720, 8200, 200, offsets_of([300, 0, 100, 200, 64], 5)),
    (720, 136, 8264, offsets_of([300, 0, 100, 200, 64], 5)),
    (1300, 4096, 1032, offsets_of([256, 700, 12, 300])),
]


def run_all(lib, tokens, n, k, off, dtype, out_dtype=None, rng=None, x=None, w=None, dy=None):
    rng = rng or np.random.default_rng(tokens * 7 + n)
    e = len(off) - 1
    x = make(rng, (tokens, k), dtype) if x is None else x
    w = make(rng, (e, n, k), dtype, 0.05) if w is None else w
    dy = make(rng, (tokens, n), dtype, 0.1) if dy is None else dy
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    x64, w64, dy64 = f64(x), f64(w), f64(dy)
    for name, got_f, ref_f, length in (
            ("forward", lambda o: lib.dmuon_expert_matmul(x, w, offs, out=o),
             lambda f, o: oe.expert_matmul(f(x64), f(w64), off, o), k),
            ("input", lambda o: lib.dmuon_expert_input_grad(dy, w, offs, out=o),
             lambda f, o: oe.expert_input_grad(f(dy64), f(w64), off, o), n)):
        keep = make(rng, (tokens, n if name == "forward" else k), dtype)
        out = keep.clone()
        assert got_f(out) is out
        ref, mag = ref_f(lambda v: v, f64(keep)), ref_f(np.abs, np.abs(f64(keep)))
        check(out, ref, mag, length, dtype, name)
        inside = np.zeros(tokens, bool)
        for _, lo, hi in oe.spans(off, tokens):
            inside[lo:hi] = True
        assert torch.equal(out[torch.from_numpy(~inside).to(DEV)], keep[torch.from_numpy(~inside).to(DEV)]), name
    for od in ([BF, F32] if dtype == BF else [F32]):
        dw = lib.dmuon_expert_weight_grad(dy, x, offs, out_dtype=od)
        longest = max(hi - lo for _, lo, hi in oe.spans(off, tokens))
        check(dw, oe.expert_weight_grad(dy64, x64, off), oe.expert_weight_grad(np.abs(dy64), np.abs(x64), off),
              longest, od, "weight")
        old = make(rng, (e, n, k), od)
        acc = old.clone()
        lib.dmuon_expert_weight_grad(dy, x, offs, out=acc, accumulate=True)
        check(acc, oe.expert_weight_grad(dy64, x64, off, f64(old)),
              oe.expert_weight_grad(np.abs(dy64), np.abs(x64), off, np.abs(f64(old))), longest + 1, od, "accumulate")


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "x".join(map(str, c[:3])) + f"-{len(c[3]) - 1}")
def test_products(lib, case, dtype):
    run_all(lib, *case, dtype)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_strided_rows_and_experts(lib, dtype):
    """Column slices (aligned and not) and weights inside a larger buffer."""
    rng = np.random.default_rng(5)
    tokens, n, k, off = 200, 72, 88, offsets_of([50, 0, 149])
    for shift in (0, 8, 3):
        x = make(rng, (tokens, k + 40), dtype)[:, shift:shift + k]
        dy = make(rng, (tokens, n + 24), dtype)[:, shift:shift + n]
        w = make(rng, (3, n + 9, k + 16), dtype, 0.05)[:, shift:shift + n, shift:shift + k]
        run_all(lib, tokens, n, k, off, dtype, rng=rng, x=x, w=w, dy=dy)
        # results with a stride leave their neighbours alone
        big = make(rng, (tokens, n + 16), dtype)
        keep = big.clone()
        offs = torch.tensor(off, dtype=torch.int32, device=DEV)
        lib.dmuon_expert_matmul(x, w, offs, out=big[:, shift:shift + n])
        ref = lib.dmuon_expert_matmul(x, w, offs)
        assert torch.equal(big[:off[-1], shift:shift + n], ref[:off[-1]])
        big[:, shift:shift + n] = keep[:, shift:shift + n]
        assert torch.equal(big, keep)


def test_broken_offsets_stay_inside(lib):
    """Offsets that decrease or leave 0..tokens are clamped as the oracle says."""
    rng = np.random.default_rng(6)
    for off in ([-7, 20, 10, 90, 5000], [60, 10, 20], [70000, 1, 2]):
        run_all(lib, 64, 48, 40, off, BF, rng=rng)


def test_no_tokens(lib):
    x = torch.zeros(0, 16, dtype=BF, device=DEV)
    w = torch.ones(2, 8, 16, dtype=BF, device=DEV)
    offs = torch.zeros(3, dtype=torch.int32, device=DEV)
    assert lib.dmuon_expert_matmul(x, w, offs).shape == (0, 8)
    dy = torch.zeros(0, 8, dtype=BF, device=DEV)
    assert lib.dmuon_expert_input_grad(dy, w, offs).shape == (0, 16)
    dw = torch.full((2, 8, 16), 3.0, dtype=F32, device=DEV)
    lib.dmuon_expert_weight_grad(dy, x, offs, out=dw, accumulate=True)
    assert (dw == 3).all()
    lib.dmuon_expert_weight_grad(dy, x, offs, out=dw)
    assert (dw == 0).all()


def test_nonfinite_rows_stay_in_their_rows(lib):
    """A NaN token reaches its own result row and its own expert's gradient only;
    rows of no expert may hold anything."""
    rng = np.random.default_rng(7)
    tokens, n, k, off = 300, 96, 160, [0, 100, 100, 290]
    x, w, dy = make(rng, (tokens, k), BF), make(rng, (3, n, k), BF), make(rng, (tokens, n), BF)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    x[120] = float("nan")
    x[290:] = float("inf")
    dy[290:] = float("nan")
    y = lib.dmuon_expert_matmul(x, w, offs)
    bad = ~torch.isfinite(y).all(dim=1)
    assert bad.nonzero().flatten().tolist() == [120]
    dw = lib.dmuon_expert_weight_grad(dy, x, offs)
    assert torch.isfinite(dw[0]).all() and (dw[1] == 0).all() and torch.isnan(dw[2]).all()
    dx = lib.dmuon_expert_input_grad(dy, w, offs)
    assert torch.isfinite(dx).all()


def test_gradients_against_differences(lib):
    """fp32 products are bilinear: a central difference of sum(y * dy) with
    step h is exact up to the rounding of y, K 2^-24 S per value, over h."""
    rng = np.random.default_rng(8)
    tokens, n, k, off = 40, 20, 36, [3, 17, 17, 40]
    x, w, dy = make(rng, (tokens, k), F32), make(rng, (3, n, k), F32), make(rng, (tokens, n), F32)
    offs = torch.tensor(off, dtype=torch.int32, device=DEV)
    dx = lib.dmuon_expert_input_grad(dy, w, offs)
    dw = lib.dmuon_expert_weight_grad(dy, x, offs)
    mag = float((f64(x).__abs__().max() * np.abs(f64(w)).max() * k))
    slack = 2 * tokens * n * np.abs(f64(dy)).max() * (k + 2) * 2.0 ** -24 * mag

    def loss():
        return float((lib.dmuon_expert_matmul(x, w, offs).double() * dy.double()).sum())

    for t, g in ((x, dx), (w, dw)):
        for _ in range(6):
            i = tuple(int(rng.integers(0, s)) for s in t.shape)
            keep = t[i].item()
            t[i] = keep + 1
            hi = loss()
            t[i] = keep - 1
            lo = loss()
            t[i] = keep
            assert abs((hi - lo) / 2 - g[i].item()) <= slack + 1e-6 * abs(g[i].item())


def test_side_stream_and_replays(lib):
    """On another stream, and captured into a graph and replayed, with other
    offsets and inputs in the same buffers: every replay equals the eager call."""
    rng = np.random.default_rng(9)
    tokens, n, k = 400, 136, 200
    x, w, dy = make(rng, (tokens, k), BF), make(rng, (4, n, k), BF), make(rng, (tokens, n), BF)
    offs = torch.tensor([0, 10, 200, 200, 390], dtype=torch.int32, device=DEV)
    y, dx, dw = torch.zeros(tokens, n, dtype=BF, device=DEV), torch.zeros(tokens, k, dtype=BF, device=DEV), \
        torch.zeros(4, n, k, dtype=F32, device=DEV)

    def go(stream=None):
        lib.dmuon_expert_matmul(x, w, offs, out=y, stream=stream)
        lib.dmuon_expert_input_grad(dy, w, offs, out=dx, stream=stream)
        lib.dmuon_expert_weight_grad(dy, x, offs, out=dw, stream=stream)

    go()
    torch.cuda.synchronize()
    want = [t.clone() for t in (y, dx, dw)]
    side = torch.cuda.Stream()
    for t in (y, dx, dw):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    go(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for new in ([0, 10, 200, 200, 390], [5, 5, 5, 300, 400], [0, 0, 0, 0, 0]):
        offs.copy_(torch.tensor(new, dtype=torch.int32))
        x.mul_(0.5)
        for t in (y, dx, dw):
            t.zero_()
        go()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, dx, dw)]
        for t in (y, dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), want)), new


def test_profile_report(lib):
    x, w = torch.ones(4, 16, dtype=BF, device=DEV), torch.ones(1, 8, 16, dtype=BF, device=DEV)
    offs = torch.tensor([0, 4], dtype=torch.int32, device=DEV)
    lib.dmuon_profile_begin()
    lib.dmuon_expert_matmul(x, w, offs)
    got = lib.dmuon_profile_end()["kernels"]["expert_bf16"]
    assert got["launches"] == 1 and got["flops"] == 2 * 4 * 8 * 16
