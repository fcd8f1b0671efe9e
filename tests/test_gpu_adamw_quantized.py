"""AdamW step with 8-bit states against the oracle.

The states follow fp32 operations that the header fixes one by one, so their
codes and scales have to be equal.  The parameter: a, b, m, r and the constants
are rounded to fp32 once each and the update goes through five more roundings
(one of them a reciprocal of 1 ulp at most): 12 2^-24 of the update's size, 2 2^-24 of
the parameter, and half a step of its type (2^-8, 2^-24) of the result."""
import numpy as np
import pytest
import torch

from oracle import adamw_quantized as oq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


@pytest.fixture(scope="module")
def lib():
    import matrix_optimizer_step_owned_amd as dm
    return dm


def codes(t):
    return t.view(torch.uint8).cpu().numpy().ravel()


def make(rng, n, dtype, gdtype, spread=2.0, first=0):
    """Device tensors of one parameter, views that begin `first` elements into a buffer."""
    g = rng.standard_normal(n) * 1e-3 * np.exp(spread * rng.standard_normal(n))
    m, r = (0.3 * g + 1e-4 * rng.standard_normal(n)).astype(np.float32), np.abs(g * (0.5 + rng.random(n))).astype(np.float32)
    (mq, ms), (rq, rs) = oq.nearest(m), oq.nearest(r)

    def place(a, dt):
        buf = torch.zeros(a.size + first, dtype=dt, device=DEV)
        buf[first:] = torch.from_numpy(a).to(DEV).to(dt)
        return buf[first:]

    f8 = lambda a: place(a, torch.uint8).view(torch.float8_e4m3fn)
    return dict(p=place(rng.standard_normal(n).astype(np.float32) * 0.02, DT[dtype]),
                g=place(g.astype(np.float32), DT[gdtype]), m=f8(mq), ms=torch.from_numpy(ms).to(DEV), r=f8(rq),
                rs=torch.from_numpy(rs).to(DEV))


def call(lib, ts, **kw):
    lib.dmuon_adamw_step_quantized(*[[t[k] for t in ts] for k in ("p", "g", "m", "ms", "r", "rs")], **kw)


def expect(s, **kw):
    f = lambda x: x.float().cpu().numpy()
    return oq.step(f(s["p"]), f(s["g"]), codes(s["m"]), f(s["ms"]), codes(s["r"]), f(s["rs"]), **kw)


def check(t, ref, dtype, old, what=""):
    p, m, r, (mq, ms), (rq, rs) = ref
    for name, got, want in (("m", codes(t["m"]), mq), ("r", codes(t["r"]), rq), ("ms", t["ms"].cpu().numpy(), ms),
                            ("rs", t["rs"].cpu().numpy(), rs)):
        assert np.array_equal(got, want), (what, name, int((got != want).sum()))
    got = t["p"].double().cpu().numpy()
    tol = 2.0 ** -24 * (12 * np.abs(p - old) + 4 * np.abs(old)) + HALF[dtype] * np.abs(p) + 1e-40
    assert (np.abs(got - p) <= tol).all(), (what, float((np.abs(got - p) / tol).max()))


@pytest.mark.parametrize("n", [1, 7, 8, 127, 128, 129, 1000, 2048, 8191, 8192, 8193, 50001])
@pytest.mark.parametrize("dtype,gdtype", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("first", [0, 1])
def test_step(lib, n, dtype, gdtype, first):
    rng = np.random.default_rng(n + first)
    t = make(rng, n, dtype, gdtype, first=first)
    for step in (1, 2, 1000):
        old = t["p"].double().cpu().numpy()
        ref = expect(t, t=step, seed=n, lr=2e-3, eps=1e-9, weight_decay=0.1)
        call(lib, [t], step=step, lr=2e-3, eps=1e-9, weight_decay=0.1, seed=n)
        check(t, ref, dtype, old, (n, step))


def test_first_steps_from_zero_states(lib):
    """States of dmuon_adamw_quantized_state against the formula without any rounding.  With e
    the distance before a step and m the formula's new value, the value that is rounded is off by
    at most b1 e, and rounding adds half a spacing: 2^-4 of it, or half of 2^-9 scales where it is
    subnormal.  sqrt(b2 r^2 + c) moves by no more than r does, and rounding at random adds up to a
    whole spacing, 2^-3 of it or 2^-9 scales.  2^-20 covers the fp32 operations."""
    rng = np.random.default_rng(3)
    p = torch.from_numpy(rng.standard_normal((37, 53)).astype(np.float32)).to(DEV)
    m, ms, r, rs = lib.dmuon_adamw_quantized_state(p)
    assert m.shape == p.shape and ms.numel() == -(-p.numel() // 128)
    m64, v64, em, er = (np.zeros(p.numel()) for _ in range(4))
    for step in range(1, 6):
        g = torch.from_numpy(rng.standard_normal((37, 53)).astype(np.float32)).to(DEV)
        lib.dmuon_adamw_step_quantized([p], [g], [m], [ms], [r], [rs], step=step, seed=1)
        g64 = g.double().cpu().numpy().ravel()
        m64, v64 = 0.9 * m64 + 0.1 * g64, 0.999 * v64 + 0.001 * g64 ** 2
        r64 = np.sqrt(v64)
        low = [np.repeat(t.double().cpu().numpy(), 128)[:p.numel()] * 2.0 ** -9 for t in (ms, rs)]
        em = 0.9 * em + (2.0 ** -4 + 2.0 ** -20) * (np.abs(m64) + 0.9 * em) + low[0] / 2 + 2.0 ** -20 * np.abs(g64)
        er = er + (2.0 ** -3 + 2.0 ** -20) * (r64 + er) + low[1]
        got_m, got_r = (oq.values(codes(q), t.cpu().numpy()).astype(np.float64) for q, t in ((m, ms), (r, rs)))
        assert (np.abs(got_m - m64) <= em).all() and (np.abs(got_r - r64) <= er).all(), step


def test_many_tensors_groups_and_skipped(lib):
    """More tensors than one launch holds, more groups than one launch holds; tensors
    without a gradient and without elements keep their place in the numbering."""
    rng = np.random.default_rng(5)
    ts = [make(rng, int(n), "bf16" if i % 3 else "f32", "bf16" if i % 2 else "f32")
          for i, n in enumerate(rng.integers(1, 3000, 97))]
    for i in (3, 50):
        ts[i]["g"] = None
    empty = torch.zeros(0, device=DEV)
    ts[7] = dict(p=empty, g=empty, m=empty.to(torch.float8_e4m3fn), ms=empty, r=empty.to(torch.float8_e4m3fn), rs=empty)
    groups = [dict(lr=1e-3 * (k + 1), betas=(0.9, 0.99 + 1e-4 * k), eps=1e-8, weight_decay=0.01 * k, step=k + 1)
              for k in range(19)]
    index = [i % 19 for i in range(97)]
    before = [{k: (v.clone() if v is not None else None) for k, v in t.items()} for t in ts]
    call(lib, ts, groups=groups, group_index=index, seed=77)
    for i, (t, b) in enumerate(zip(ts, before)):
        if i == 7:
            continue
        if b["g"] is None:
            assert torch.equal(t["p"], b["p"]) and torch.equal(t["m"].view(torch.uint8), b["m"].view(torch.uint8))
            continue
        h = dict(groups[index[i]])
        ref = expect(b, t=h.pop("step"), seed=77, place=i, **h)
        check(t, ref, "bf16" if i % 3 else "f32", b["p"].double().cpu().numpy(), i)


def test_nothing_outside_the_tensor(lib):
    """Odd tensors back to back in flat buffers: one stepped alone leaves its neighbours."""
    rng = np.random.default_rng(6)
    n, a, b = 1000, 301, 680
    flat = make(rng, n, "bf16", "bf16")
    view = dict(p=flat["p"][a:b], g=flat["g"][a:b], m=flat["m"][a:b], r=flat["r"][a:b], ms=flat["ms"][2:5], rs=flat["rs"][2:5])
    before = {k: v.clone() for k, v in flat.items()}
    old = view["p"].double().cpu().numpy()
    ref = expect(view, t=4)
    call(lib, [view], step=4)
    check(view, ref, "bf16", old)
    for k in ("p", "g"):
        assert torch.equal(flat[k][:a], before[k][:a]) and torch.equal(flat[k][b:], before[k][b:])
    for k in ("m", "r"):
        x, y = codes(flat[k]), codes(before[k])
        assert np.array_equal(x[:a], y[:a]) and np.array_equal(x[b:], y[b:])
    for k in ("ms", "rs"):
        assert torch.equal(flat[k][:2], before[k][:2]) and torch.equal(flat[k][5:], before[k][5:])


def test_not_finite_and_extreme_gradients(lib):
    rng = np.random.default_rng(8)
    t = make(rng, 128 * 6, "f32", "f32")
    g = t["g"]
    g[5], g[128 + 3], g[256 + 9] = float("nan"), float("inf"), -float("inf")
    g[3 * 128:4 * 128] = 0
    g[4 * 128:5 * 128] *= 1e-30          # squares below fp32
    g[5 * 128:] *= 1e15
    t["m"].view(torch.uint8)[3 * 128:4 * 128] = 0
    t["r"].view(torch.uint8)[3 * 128:4 * 128] = 0
    with np.errstate(all="ignore"):
        ref = expect(t, t=2, eps=1e-8)
    old = t["p"].double().cpu().numpy()
    call(lib, [t], step=2, eps=1e-8)
    ms, rs = t["ms"].cpu().numpy(), t["rs"].cpu().numpy()
    assert not np.isfinite(ms[:3]).any() and not np.isfinite(rs[:3]).any()
    assert np.isfinite(ms[3:]).all() and np.isfinite(rs[3:]).all()
    tail = slice(3 * 128, None)
    p, _, _, (mq, mscale), (rq, rscale) = ref
    assert np.array_equal(codes(t["m"])[tail], mq[tail]) and np.array_equal(codes(t["r"])[tail], rq[tail])
    assert np.array_equal(ms[3:], mscale[3:]) and np.array_equal(rs[3:], rscale[3:])
    got = t["p"].double().cpu().numpy()
    bad = np.zeros(got.size, bool)
    bad[[5, 128 + 3, 256 + 9]] = True
    assert np.isfinite(got[~bad]).all()          # neighbours keep their step
    tol = 2.0 ** -24 * (12 * np.abs(p - old) + 6 * np.abs(old)) + 1e-40
    assert (np.abs(got - p)[~bad] <= tol[~bad]).all()


def test_repeats_and_seeds(lib):
    rng = np.random.default_rng(9)
    base = make(rng, 40000, "bf16", "bf16")
    runs = []
    for seed, step in ((1, 9), (1, 9), (2, 9), (1, 10)):
        t = {k: v.clone() for k, v in base.items()}
        call(lib, [t], step=step, seed=seed)
        runs.append(codes(t["r"]))
    assert np.array_equal(runs[0], runs[1])
    for other in runs[2:]:
        assert 0.001 < np.mean(runs[0] != other) < 0.9


def test_random_rounding_is_unbiased(lib):
    """One value half, a tenth, a hundredth of the way between two neighbours: the share that goes up, over
    n elements of independent 16-bit numbers, within five standard deviations."""
    n = 128 * 512
    for part in (0.5, 0.1, 0.01):
        r = np.full(n, np.float32(16 + 2 * part))       # spacing 2 where 448 is the block's largest
        r[::128] = 448
        # beta2 = 0 makes r' = |g|
        p = torch.zeros(n, device=DEV)
        g = torch.from_numpy(r).to(DEV)
        m, ms, q, qs = lib.dmuon_adamw_quantized_state(p)
        lib.dmuon_adamw_step_quantized([p], [g], [m], [ms], [q], [qs], step=1, betas=(0.9, 0.0), seed=123)
        got = oq.values(codes(q), qs.cpu().numpy()).reshape(-1, 128)[:, 1:]
        assert set(np.unique(got)) == {16.0, 18.0}
        want = float(np.float32(16 + 2 * part) - 16) / 2
        share, k = np.mean(got == 18), got.size
        assert abs(share - want) <= 5 * np.sqrt(want * (1 - want) / k) + 2.0 ** -16


def test_graph_stream_and_interop(lib):
    """Captured and replayed next to eager work, on a stream of its own; states are the blocks of
    dmuon_dequantize_blocks."""
    rng = np.random.default_rng(10)
    base = make(rng, 128 * 300, "f32", "bf16")
    t, e = ({k: v.clone() for k, v in base.items()} for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(lib, [t], step=5)
    torch.cuda.synchronize()
    for _ in range(4):
        graph.replay()
        torch.cuda.synchronize()
        call(lib, [e], step=5, stream=side)
        side.synchronize()
        assert torch.equal(t["p"], e["p"]) and np.array_equal(codes(t["r"]), codes(e["r"]))
        assert np.array_equal(codes(t["m"]), codes(e["m"])) and torch.equal(t["rs"], e["rs"])
    got = lib.dmuon_dequantize_blocks(e["m"].view(-1, 128), e["ms"].view(-1, 1), dtype=torch.float32)
    assert np.array_equal(got.cpu().numpy().ravel(), oq.values(codes(e["m"]), e["ms"].cpu().numpy()))


def test_long_tensor(lib):
    """Past 2^31 elements: the last ones, and the blocks around 2^31."""
    n = (1 << 31) + 5000
    p = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    m, ms, r, rs = lib.dmuon_adamw_quantized_state(p)
    spots = [0, (1 << 31) - 8192, (1 << 31), n - 1000]
    rng = np.random.default_rng(11)
    for s in spots:
        g[s:s + 1000] = torch.from_numpy(rng.standard_normal(1000).astype(np.float32)).to(DEV).bfloat16()
    lib.dmuon_adamw_step_quantized([p], [g], [m], [ms], [r], [rs], step=1, seed=4)
    u_of = lambda s, k: _randoms_at(4, 1, 0, s, k)
    for s in spots:
        lo = s // 128 * 128
        k = min(n - lo, 1280)
        g32 = g[lo:lo + k].float().cpu().numpy()
        mm, rr = np.float32(0.1) * g32, np.sqrt(np.float32(1 - 0.999) * (g32 * g32))
        mq, msc = oq.nearest(mm)
        rq, rsc = oq.at_random(rr, u_of(lo, k))
        assert np.array_equal(codes(m[lo:lo + k]) & 127, mq & 127)
        assert np.array_equal(codes(r[lo:lo + k]), rq)
        assert np.array_equal(ms[lo // 128:lo // 128 + msc.size].cpu().numpy(), msc)
        assert np.array_equal(rs[lo // 128:lo // 128 + rsc.size].cpu().numpy(), rsc)
    assert int((p != 0).sum()) >= 3900


def _randoms_at(seed, step, place, first, n):
    mix, U = oq.mix, np.uint64
    key = mix(mix(mix(seed) + U(step)) + U(place))
    i = np.arange(first, first + n, dtype=np.uint64)
    w = mix(mix(key + i // U(8192)) + i // U(2) % U(4096))
    return np.where(i % U(2) == 0, w & U(0xffff), w >> U(16))
