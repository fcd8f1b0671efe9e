"""The expert layer for a few tokens against the oracle (the bound is derived in
oracle.rows.layer; y's own rounding to bf16 is 2^-8 of it), and the 8-bit set as
it is used: a step, quantised weights, prompts and single tokens."""
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


def make(rng, tokens, experts, top_k, n, k, int8, distinct=True):
    s = dict(x=torch.from_numpy(rng.standard_normal((tokens, k)).astype(np.float32)).to(DEV).to(BF))
    pick = lambda: rng.choice(experts, top_k, replace=not distinct or top_k > experts)
    ids = np.stack([pick() for _ in range(tokens)]) if tokens else np.zeros((0, top_k))
    s["ids"] = torch.from_numpy(ids.astype(np.int32)).to(DEV)
    s["gates"] = torch.from_numpy(rng.random((tokens, top_k)).astype(np.float32)).to(DEV)
    s["in_scale"] = s["out_scale"] = None
    for name, shape in (("w_in", (experts, 2 * n, k)), ("w_out", (experts, k, n))):
        if int8:
            s[name] = torch.from_numpy(rng.integers(-128, 128, shape, dtype=np.int8)).to(DEV)
            s[name[2:] + "_scale"] = torch.from_numpy((rng.random(shape[:2]) + 0.5).astype(np.float32) / 2000).to(DEV)
        else:
            s[name] = torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * 0.05).to(DEV).to(BF)
    return s


def call(lib, s, **kw):
    return lib.dmuon_expert_layer(s["x"], s["ids"], s["gates"], s["w_in"], s["w_out"], in_scale=s["in_scale"],
                                  out_scale=s["out_scale"], **kw)


def expect(s):
    f = lambda t: t.double().cpu().numpy()
    w_in, w_out = f(s["w_in"]), f(s["w_out"])
    if s["in_scale"] is not None:
        w_in, w_out = w_in * f(s["in_scale"])[..., None], w_out * f(s["out_scale"])[..., None]
    return orow.layer(f(s["x"]), s["ids"].cpu().numpy(), f(s["gates"]), w_in, w_out)


def check(got, s, what=""):
    y, err = expect(s)
    got = got.double().cpu().numpy()
    tol = err + 2.0 ** -8 * (np.abs(y) + err) + 1e-38
    assert np.isfinite(got).all() and (np.abs(got - y) <= tol).all(), (what, float((np.abs(got - y) / tol).max()))


CASES = [(1, 1, 1, 1, 1), (1, 4, 2, 16, 32), (2, 3, 3, 8, 8), (5, 16, 3, 33, 100), (7, 5, 2, 17, 65), (16, 8, 4, 48, 136),
         (17, 6, 2, 64, 256), (33, 4, 3, 40, 72), (64, 5, 2, 96, 264), (64, 2, 1, 24, 16), (3, 64, 8, 256, 512),
         (20, 130, 6, 32, 64), (1, 3, 2, 1000, 520), (4, 4, 4, 520, 1040), (9, 4096, 2, 8, 16), (50, 3, 2, 515, 129)]


@pytest.mark.parametrize("tokens,experts,top_k,n,k", CASES)
@pytest.mark.parametrize("int8", [False, True])
def test_layer(lib, tokens, experts, top_k, n, k, int8):
    s = make(np.random.default_rng(tokens + n + k), tokens, experts, top_k, n, k, int8)
    check(call(lib, s), s)


@pytest.mark.parametrize("int8", [False, True])
def test_layer_strides_and_guards(lib, int8):
    """Strided rows, experts apart, a workspace and a result between guards, another stream."""
    rng = np.random.default_rng(1)
    for n, k in ((48, 64), (45, 61)):
        s = make(rng, 11, 6, 2, n, k, int8)
        want = call(lib, s)
        pad = 16 if n % 16 == 0 else 3
        t = dict(s)
        for name in ("x", "w_in", "w_out"):
            big = torch.ones(s[name].shape[:-1] + (s[name].shape[-1] + pad,), dtype=s[name].dtype, device=DEV) * 77
            big[..., :s[name].shape[-1]] = s[name]
            t[name] = big[..., :s[name].shape[-1]]
        out = torch.full((13, k + pad), 5.0, dtype=BF, device=DEV)
        d = lib.dmuon_expert_layer_t(tokens=11, n=n, k=k, experts=6, top_k=2)
        need = lib._lib.dmuon_expert_layer_workspace_size(d)
        ws = torch.full((need + 64,), 7, dtype=torch.uint8, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        call(lib, t, out=out[1:12, :k], workspace=ws[32:32 + need], stream=side)
        side.synchronize()
        assert torch.equal(out[1:12, :k], want)
        check(want, s)
        assert (out[0] == 5).all() and (out[12] == 5).all() and (out[:, k:] == 5).all()
        assert (ws[:32] == 7).all() and (ws[32 + need:] == 7).all()


@pytest.mark.parametrize("int8", [False, True])
def test_layer_ids(lib, int8):
    """Picks of nobody, a token without picks, the same expert twice, all tokens on one expert."""
    rng = np.random.default_rng(2)
    s = make(rng, 40, 7, 4, 40, 72, int8, distinct=False)
    ids = s["ids"]
    ids[0] = -1
    ids[1] = torch.tensor([7, 100000, -2 ** 31, 3], device=DEV)
    ids[2] = 5
    ids[3] = torch.tensor([2, 2, 6, 2], device=DEV)
    got = call(lib, s)
    check(got, s)
    assert (got[0] == 0).all()
    ids[:] = 4
    check(call(lib, s), s)
    ids[:] = -1
    assert (call(lib, s) == 0).all()
    for dt in ("ids", "gates"):
        s[dt] = s[dt][:0].contiguous()
    s["x"] = s["x"][:0]
    assert call(lib, s).shape == (0, 72)


@pytest.mark.parametrize("int8", [False, True])
def test_layer_not_finite(lib, int8):
    """A token's NaN or Inf stays its own; a weight's reaches its expert's tokens only."""
    rng = np.random.default_rng(3)
    s = make(rng, 24, 6, 2, 32, 64, int8)
    s["ids"] = torch.stack((torch.arange(24) % 5, torch.full((24,), 5)), 1).int().to(DEV)
    s["ids"][1::5, 1] = 0                      # tokens of expert 1: 1 and 0
    clean = call(lib, s)
    s["x"][3, 7] = float("nan")
    s["x"][10, 0] = float("inf")
    got = call(lib, s)
    keep = torch.ones(24, dtype=torch.bool, device=DEV)
    keep[3] = keep[10] = False
    assert torch.equal(got[keep], clean[keep]) and not torch.isfinite(got[3]).all() and not torch.isfinite(got[10]).all()
    for name in ("w_in", "w_out"):
        t = make(np.random.default_rng(3), 24, 6, 2, 32, 64, int8)
        t["ids"] = s["ids"]
        if int8:
            t[name[2:] + "_scale"][1, 9] = float("nan")
        else:
            t[name][1, 9, 5] = float("nan")
        got = call(lib, t)
        hit = (t["ids"] == 1).any(1)
        assert torch.equal(got[~hit], clean[~hit]) and torch.isnan(got[hit]).any(1).all()


@pytest.mark.parametrize("int8", [False, True])
def test_layer_inf_is_not_nan(lib, int8):
    """An Inf in x with weights of one sign: G x and U x are Inf, and so is y, not NaN, also where
    the sums end inside the last loads."""
    for n, k in ((48, 80), (48, 64), (45, 61), (8, 16)):
        s = make(np.random.default_rng(1), 5, 3, 2, n, k, int8)
        for name in ("w_in", "w_out"):
            s[name] = s[name].float().abs().clamp(1, 127).to(s[name].dtype)      # 128 is no int8
        s["x"] = s["x"].abs()
        s["x"][2, k - 1] = s["x"][4, 0] = float("inf")
        got = call(lib, s)
        assert torch.isfinite(got[[0, 1, 3]]).all()
        assert (got[[2, 4]] == float("inf")).all()


def test_layer_many_tiles(lib):
    """More tiles than waves: several rounds per block, and one wave, two or all per tile.  The reference
    and its bound are those of oracle.rows.layer, an expert at a time in float64 on the GPU."""
    u = 2.0 ** -24
    for tokens, experts, top_k, n, k, int8 in ((3, 40, 8, 4096, 1040, False), (60, 300, 5, 1030, 272, True),
                                               (64, 256, 8, 512, 528, False), (64, 4, 2, 2048, 1024, True)):
        gen = torch.Generator(device=DEV).manual_seed(n)
        s = make(np.random.default_rng(2), tokens, experts, top_k, 1, 1, int8)
        s["x"] = torch.randn(tokens, k, generator=gen, device=DEV).to(BF)
        for name, shape in (("w_in", (experts, 2 * n, k)), ("w_out", (experts, k, n))):
            w = torch.randn(shape, generator=gen, device=DEV) * 0.05
            s[name] = (w * 500).round().clamp(-127, 127).to(torch.int8) if int8 else w.to(BF)
            if int8:
                s[name[2:] + "_scale"] = torch.rand(shape[:2], generator=gen, device=DEV) / 500
        got = call(lib, s).double()
        y, err, mag = (torch.zeros(tokens, k, dtype=torch.float64, device=DEV) for _ in range(3))
        x = s["x"].double()
        for e in range(experts):
            gate = (s["gates"].double() * (s["ids"] == e)).sum(1, keepdim=True)
            w_in, w_out = s["w_in"][e].double(), s["w_out"][e].double()
            if int8:
                w_in, w_out = w_in * s["in_scale"][e].double()[:, None], w_out * s["out_scale"][e].double()[:, None]
            up, size = x @ w_in.T.contiguous(), (k + 8) * u * (x.abs() @ w_in.abs().T.contiguous())
            a, b, da, db = up[:, :n], up[:, n:], size[:, :n], size[:, n:]
            act = torch.nn.functional.silu(a)
            h = gate * act * b
            dh = gate.abs() * (1.1 * da * (b.abs() + db) + act.abs() * db) + h.abs() * (2 * a.abs() + 16) * 2 * u
            dh += 2.0 ** -16 * (h.abs() + dh) + 2.0 ** -133
            dh *= gate != 0
            y += h @ w_out.T.contiguous()
            err += dh @ w_out.abs().T.contiguous()
            mag += (h.abs() + dh) @ w_out.abs().T.contiguous()
        err += (2 * n * top_k + 8) * u * mag
        tol = err + 2.0 ** -8 * (y.abs() + err) + 1e-38
        assert bool(torch.isfinite(got).all()) and bool(((got - y).abs() <= tol).all()), float(((got - y).abs() / tol).max())


def test_layer_graph_two_streams(lib):
    """Two captured calls with workspaces of their own, replayed next to eager ones."""
    rng = np.random.default_rng(4)
    a, b = make(rng, 3, 8, 2, 256, 512, False), make(rng, 20, 8, 2, 256, 512, True)
    want = [call(lib, a), call(lib, b)]
    outs = [torch.zeros_like(w) for w in want]
    wss = [torch.empty(1 << 22, dtype=torch.uint8, device=DEV) for s in (a, b)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            for s, o, w in zip((a, b), outs, wss):
                call(lib, s, out=o, workspace=w)
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        graph.replay()
        again = [call(lib, a), call(lib, b)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(want, outs, again))


def test_layer_repeats_bit_for_bit(lib):
    """Blocks that split the same columns join in a fixed order: many calls in a row, inputs in turn in one
    workspace, with copies on another stream beside them."""
    side, big = torch.cuda.Stream(), torch.zeros(1 << 26, device=DEV)
    copy = torch.empty_like(big)
    for args in ((5, 16, 3, 515, 1000, False), (20, 32, 4, 256, 512, True), (40, 8, 2, 512, 256, False)):
        ss = [make(np.random.default_rng(i), *args) for i in range(2)]
        want = [call(lib, s) for s in ss]
        ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
        wrong = torch.zeros((), dtype=torch.int64, device=DEV)
        for i in range(200):
            if i % 20 == 0:
                with torch.cuda.stream(side):
                    copy.copy_(big)
            wrong += (call(lib, ss[i % 2], workspace=ws) != want[i % 2]).sum()
        assert int(wrong) == 0


def test_profile_report(lib):
    """The kernels' names and launches in a profile."""
    s = make(np.random.default_rng(3), 5, 16, 3, 515, 1000, True)
    call(lib, s)
    x = torch.randn(40, 512, device=DEV)
    p, st = x.clone(), lib.dmuon_adamw_quantized_state(x)
    lib.dmuon_profile_begin()
    call(lib, s)
    q, sc = lib.dmuon_quantize_rows(x)
    lib.dmuon_dequantize_rows(q, sc)
    lib.dmuon_row_matmul(q, sc, q, sc)
    lib.dmuon_adamw_step_quantized([p], [x], [st[0]], [st[1]], [st[2]], [st[3]], step=1)
    got = lib.dmuon_profile_end()["kernels"]
    for name in ("layer_in", "layer_out", "quantize_rows", "dequantize_rows", "int8_matmul", "adamw8"):
        assert got[name]["launches"] == 1, name


def test_layer_far_weights(lib):
    """Experts more than 2^32 bytes apart."""
    rng = np.random.default_rng(5)
    s = make(rng, 3, 3, 2, 32, 64, False)
    want = call(lib, s)
    far = (1 << 31) + 64
    store = torch.zeros(3 * far, dtype=BF, device=DEV)
    for name, first in (("w_in", 0), ("w_out", 8192)):
        v = store[first:].as_strided(s[name].shape, (far - 4096, s[name].shape[2], 1))
        v.copy_(s[name])
        s[name] = v
    assert torch.equal(call(lib, s), want)


def test_step_quantise_prompt_and_tokens(lib):
    """A layer's life: its weights take a step with 8-bit states, are quantised by output
    channel, and serve prompts (8-bit products with the gated activation between) and single tokens
    from the same integers.  Bounds: the tokens' path as above with the dequantised weights; the
    prompt's against float64 over the integers that it was given."""
    rng = np.random.default_rng(6)
    e, n, k, tokens, top_k = 4, 96, 128, 24, 2
    s = make(rng, tokens, e, top_k, n, k, False)
    for name in ("w_in", "w_out"):
        w = s[name]
        state = lib.dmuon_adamw_quantized_state(w)
        old = w.clone()
        g = torch.from_numpy(rng.standard_normal(w.shape).astype(np.float32)).to(DEV).to(BF)
        lib.dmuon_adamw_step_quantized([w], [g], [state[0]], [state[1]], [state[2]], [state[3]], step=1, lr=0.02)
        assert (torch.sign(old.float() - w.float()) == torch.sign(g.float()))[g != 0].float().mean() > 0.95
        s[name], s[name[2:] + "_scale"] = lib.dmuon_quantize_rows(w)
    check(call(lib, s), s)
    # the same tokens as a prompt: sorted by expert, one row per pick
    order = torch.argsort(s["ids"].flatten(), stable=True)
    token = order // top_k
    off = torch.cumsum(torch.bincount(s["ids"].flatten(), minlength=e), 0)
    offsets = torch.cat((torch.zeros(1, dtype=off.dtype, device=DEV), off)).int()
    xq, xs = lib.dmuon_quantize_rows(s["x"][token])
    up = lib.dmuon_row_matmul(xq, xs, s["w_in"], s["in_scale"], offsets=offsets, out_dtype=F32)
    hq, hs = lib.dmuon_quantize_rows(up, activation="swiglu")
    down = lib.dmuon_row_matmul(hq, hs, s["w_out"], s["out_scale"], offsets=offsets, out_dtype=F32)
    c = lambda t: t.cpu().numpy()
    off_h = [int(v) for v in offsets]
    ref_up = orow.matmul(c(xq), c(xs), c(s["w_in"]), c(s["in_scale"]), off_h, np.zeros(up.shape))
    assert (np.abs(c(up) - ref_up) <= 4 * 2.0 ** -24 * np.abs(ref_up) + 1e-38).all()
    h = orow.swiglu(c(up))
    assert (np.abs(c(hq) * c(hs)[:, None].astype(np.float64) - h) <= 0.501 * c(hs)[:, None]).all()
    ref_down = orow.matmul(c(hq), c(hs), c(s["w_out"]), c(s["out_scale"]), off_h, np.zeros(down.shape))
    assert (np.abs(c(down) - ref_down) <= 4 * 2.0 ** -24 * np.abs(ref_down) + 1e-38).all()
    # both paths are the same layer: they differ by the 8-bit rounding of x and of the gated
    # activation, at most half a scale per value each; here only that they agree to a few per cent
    y = torch.zeros(tokens, k, device=DEV).index_add_(0, token, down * s["gates"].flatten()[order][:, None])
    few = call(lib, s).float()
    assert float((y - few).norm() / few.norm()) < 0.05
