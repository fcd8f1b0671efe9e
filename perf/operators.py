"""The measured cases of the expert-layer operators: the matrix products of
experts with ragged token counts (forward, input gradient, weight gradient),
the quantisation of activations and weights to 8-bit floating point with one
scale per block of 128, and the matrix product of such operands.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges,
``prepare(case, seed)`` makes what a training or serving program holds before
the call, ``run(state)`` makes one pass: with ``own`` false in plain torch
operations, with ``own`` true through the library.  ``exact`` computes the
same outputs in float64.
"""
import math

import torch

own = False

BLOCK = 128
E4M3_MAX, E5M2_MAX = 448.0, 57344.0
SCALE_MIN = 2.0 ** -126        # smallest scale of a block (an all-zero block has it)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
Q8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
Q8_MAX = {"e4m3": E4M3_MAX, "e5m2": E5M2_MAX}
DEV = "cuda"


def listed():
    return [
        # serving, one token of each of five sequences: a few experts of a
        # small layer are read for one row each; launch latency counts
        dict(name="experts decode", op="forward", experts=16, tokens=5, n=512, k=1024, dtype="bf16", tail=0, skew=1.0),
        # serving a batch through an 8B-sized expert block: every touched
        # expert's weights are read once, HBM is the bound
        dict(name="experts serve batch", op="forward", experts=8, tokens=64, n=14336, k=4096, dtype="bf16", tail=0,
             skew=0.5),
        # training, many small experts, uneven counts, rows of padding behind
        # the last expert's
        dict(name="experts forward", op="forward", experts=32, tokens=16384, n=2048, k=4096, dtype="bf16", tail=77,
             skew=1.0),
        # training, few wide experts: gradient of the layer's input
        dict(name="experts input gradient", op="input_grad", experts=8, tokens=8191, n=14336, k=4096, dtype="bf16",
             tail=0, skew=0.5),
        # training, few wide experts: gradient of the weights, as the Muon
        # step reads it
        dict(name="experts weight gradient", op="weight_grad", experts=8, tokens=8192, n=4096, k=14336, dtype="bf16",
             out="bf16", tail=0, skew=0.5),
        # single precision, odd sizes, experts without tokens
        dict(name="experts weight gradient f32", op="weight_grad", experts=24, tokens=3001, n=1000, k=515, dtype="f32",
             out="f32", tail=3, skew=2.0),
        # activations of a training step, both orientations: rows feed the
        # forward product, columns the weight gradient
        dict(name="quantise activations", op="quantise", batch=1, rows=8192, cols=14336, block_rows=1, dtype="bf16",
             fmt="e4m3", transposed=True),
        # the experts' weights after an update, one scale per 128 x 128
        dict(name="quantise weights", op="quantise", batch=8, rows=1024, cols=4096, block_rows=128, dtype="bf16",
             fmt="e4m3", transposed=False),
        # serving, seven sequences through one projection
        dict(name="fp8 decode", op="fp8", m=7, n=14336, k=4096, experts=0, b_rows=128, fmt="e4m3", out="bf16", skew=0.0),
        # training, forward of a projection
        dict(name="fp8 forward", op="fp8", m=8192, n=14336, k=4096, experts=0, b_rows=128, fmt="e4m3", out="bf16",
             skew=0.0),
        # training, weight gradient: tokens are summed, a scale per 128 of
        # them on both sides, gradients in the wide-range format
        dict(name="fp8 weight gradient", op="fp8", m=4096, n=4096, k=8190, experts=0, b_rows=1, fmt="e5m2", out="f32",
             skew=0.0),
        # training or prefill: the experts' product on quantised operands
        dict(name="fp8 experts", op="fp8", m=8192, n=4096, k=2048, experts=16, b_rows=128, fmt="e4m3", out="bf16",
             skew=1.0),
    ]


MAX_FLOPS = 2.0 * 8192 * 14336 * 4096      # the largest listed product
MAX_ELEMS = 8 * 14336 * 4096               # the largest listed tensor


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm: any number of tokens."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer's width, even over its logarithm: most are multiples of 128 or
    of 16, one in five is any number."""
    v, kind = _size(rng, lo, hi), rng.random()
    unit = 128 if kind < 0.5 and v >= 128 else 16 if kind < 0.8 and v >= 16 else 1
    return v // unit * unit


def draw(rng):
    while True:
        op = rng.choice(["forward", "input_grad", "weight_grad", "quantise", "fp8", "fp8"])
        if op == "quantise":
            c = dict(op=op, batch=rng.choice([1, 1, 2, 8]), rows=_size(rng, 1, 14336), cols=_width(rng, 16, 14336),
                     block_rows=rng.choice([1, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                     fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), transposed=rng.random() < 0.5)
            if 2 ** 12 <= c["batch"] * c["rows"] * c["cols"] <= 8192 * 14336:
                return c
            continue
        if op == "fp8":
            experts = rng.choice([0, 0, 4, 16, 61])
            c = dict(op=op, m=_size(rng, 1, 8192), n=_width(rng, 16, 14336), k=_width(rng, 32, 14336), experts=experts,
                     b_rows=128 if experts else rng.choice([1, 128]), fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                     out=rng.choice(["bf16", "bf16", "f32"]), skew=rng.choice([0.0, 0.5, 1.0, 2.0]))
            if 2.0 * c["m"] * c["n"] * c["k"] <= MAX_FLOPS and max(1, experts) * c["n"] * c["k"] <= MAX_ELEMS // 2:
                return c
            continue
        c = dict(op=op, experts=rng.choice([1, 4, 8, 24, 64, 130]), tokens=_size(rng, 1, 16384),
                 n=_width(rng, 16, 14336), k=_width(rng, 16, 14336), dtype=rng.choice(["bf16", "bf16", "bf16", "f32"]),
                 tail=rng.choice([0, 0, 1, 200]), skew=rng.choice([0.0, 0.5, 1.0, 2.0]))
        if op == "weight_grad":
            c["out"] = rng.choice(["bf16", "f32"]) if c["dtype"] == "bf16" else "f32"
        top = MAX_FLOPS / (8 if c["dtype"] == "f32" else 1)
        if 2.0 * c["tokens"] * c["n"] * c["k"] <= top and c["experts"] * c["n"] * c["k"] <= MAX_ELEMS // 2:
            return c


def _counts(g, experts, tokens, skew):
    """Tokens per expert: a routing with popular and unpopular experts (the
    popularity's logarithm is normal with deviation `skew`)."""
    p = torch.exp(skew * torch.randn(experts, generator=g, dtype=torch.float64))
    picks = torch.multinomial(p, tokens, replacement=True, generator=g)
    return torch.bincount(picks, minlength=experts)


def _normal(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _outliers(x, gen):
    """A few columns thirty times as large, as activations have them."""
    cols = torch.randint(0, x.shape[-1], (max(1, x.shape[-1] // 256),), generator=gen, device=DEV)
    x[..., cols] *= 30
    return x


def _to_blocks(x, block_rows, fmt):
    """Values (b, r, c) -> (8-bit values, fp32 scale per block of block_rows x
    128), in fp32: scale = amax / largest value of the format, x * (1/scale)
    rounded to nearest even."""
    b, r, c = x.shape
    pr, pc = -r % block_rows, -c % BLOCK
    xb = torch.nn.functional.pad(x.float(), (0, pc, 0, pr))
    xb = xb.view(b, (r + pr) // block_rows, block_rows, (c + pc) // BLOCK, BLOCK)
    scale = (xb.abs().amax(dim=(2, 4)) / Q8_MAX[fmt]).clamp_min(SCALE_MIN)
    q = (xb * (1.0 / scale)[:, :, None, :, None]).to(Q8[fmt])
    return q.view(b, r + pr, c + pc)[:, :r, :c].contiguous(), scale


def _values(q, scale, block_rows):
    """fp32 values that (q, scale) stand for."""
    s = scale.repeat_interleave(BLOCK, -1)[..., :q.shape[-1]]
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, -2)[..., :q.shape[-2], :]
    return q.float() * s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "quantise":
        x = _outliers(_normal(gen, (case["batch"], case["rows"], case["cols"]), 0.5, DT[case["dtype"]]), gen)
        s.update(x=x if case["batch"] > 1 else x[0])
        b, r, c, br = case["batch"], case["rows"], case["cols"], case["block_rows"]
        lead = (b,) if b > 1 else ()
        s["q"] = torch.empty(lead + (r, c), dtype=Q8[case["fmt"]], device=DEV)
        s["scale"] = torch.empty(lead + (-(-r // br), -(-c // BLOCK)), dtype=torch.float32, device=DEV)
        s["qt"] = s["scale_t"] = None
        if case["transposed"]:
            s["qt"] = torch.empty(lead + (c, r), dtype=Q8[case["fmt"]], device=DEV)
            s["scale_t"] = torch.empty(lead + (-(-c // br), -(-r // BLOCK)), dtype=torch.float32, device=DEV)
        return s
    if op == "fp8":
        m, n, k, e = case["m"], case["n"], case["k"], case["experts"]
        x = _outliers(_normal(gen, (1, m, k), 0.5, torch.float32), gen)
        a, a_scale = _to_blocks(x, 1, case["fmt"])
        w = _normal(gen, (max(1, e), n, k), 0.02, torch.float32)
        b, b_scale = _to_blocks(w, case["b_rows"], "e4m3")
        s.update(a=a[0], a_scale=a_scale[0], b=b if e else b[0], b_scale=b_scale if e else b_scale[0])
        s["c"] = torch.zeros(m, n, dtype=DT[case["out"]], device=DEV)
        s["bounds"] = s["offsets"] = None
        if e:
            bounds = [0] + torch.cumsum(_counts(host, e, m, case["skew"]), 0).tolist()
            s["bounds"], s["offsets"] = bounds, torch.tensor(bounds, dtype=torch.int32, device=DEV)
        return s
    e, t, n, k, dt = case["experts"], case["tokens"], case["n"], case["k"], DT[case["dtype"]]
    bounds = [0] + torch.cumsum(_counts(host, e, t, case["skew"]), 0).tolist()
    s["bounds"], s["offsets"] = bounds, torch.tensor(bounds, dtype=torch.int32, device=DEV)
    rows = t + case["tail"]
    if op != "input_grad":
        s["x"] = _outliers(_normal(gen, (rows, k), 0.5, dt), gen)
    if op != "weight_grad":
        s["w"] = _normal(gen, (e, n, k), 0.02, dt)
    if op != "forward":
        s["dy"] = _normal(gen, (rows, n), 1e-3, dt)
    if op == "weight_grad":
        s["out"] = torch.zeros(e, n, k, dtype=DT[case["out"]], device=DEV)
    else:
        s["out"] = torch.zeros(rows, n if op == "forward" else k, dtype=dt, device=DEV)
    return s


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quantise":
        x = s["x"] if s["x"].dim() == 3 else s["x"][None]
        q, scale = _to_blocks(x, s["block_rows"], s["fmt"])
        got = [q, scale]
        if s["transposed"]:
            got += _to_blocks(x.transpose(1, 2), s["block_rows"], s["fmt"])
        return [v if s["x"].dim() == 3 else v[0] for v in got]
    if op == "fp8":
        a = _values(s["a"], s["a_scale"], 1)
        if s["bounds"] is None:
            return (a @ _values(s["b"], s["b_scale"], s["b_rows"]).T).to(s["c"].dtype)
        bounds = s["bounds"]
        return torch.cat([a[lo:hi] @ _values(s["b"][e], s["b_scale"][e], s["b_rows"]).T
                          for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])) if hi > lo]).to(s["c"].dtype)
    spans = [(e, lo, hi) for e, (lo, hi) in enumerate(zip(s["bounds"], s["bounds"][1:]))]
    out = s["out"]
    if op == "weight_grad":
        return torch.stack([s["dy"][lo:hi].float().T @ s["x"][lo:hi].float() for _, lo, hi in spans]).to(out.dtype)
    if op == "forward":
        parts = [s["x"][lo:hi].float() @ s["w"][e].float().T for e, lo, hi in spans if hi > lo]
    else:
        parts = [s["dy"][lo:hi].float() @ s["w"][e].float() for e, lo, hi in spans if hi > lo]
    out[:s["bounds"][-1]] = torch.cat(parts).to(out.dtype)
    return out


def _run_own(s):
    import matrix_optimizer_step_owned_amd as dm
    op = s["op"]
    if op == "quantise":
        got = dm.dmuon_quantize_blocks(s["x"], block_rows=s["block_rows"], fmt=s["fmt"], q=s["q"], scale=s["scale"],
                                       qt=s["qt"], scale_t=s["scale_t"])
        return [v for v in got if v is not None]
    if op == "fp8":
        return dm.dmuon_block_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], block_rows=s["b_rows"],
                                     offsets=s["offsets"], out=s["c"])
    if op == "forward":
        return dm.dmuon_expert_matmul(s["x"], s["w"], s["offsets"], out=s["out"])
    if op == "input_grad":
        return dm.dmuon_expert_input_grad(s["dy"], s["w"], s["offsets"], out=s["out"])
    return dm.dmuon_expert_weight_grad(s["dy"], s["x"], s["offsets"], out=s["out"])


def _touched(case):
    """Experts that get a token, as expected over routings: with t tokens and
    e equally popular experts e (1 - (1 - 1/e)^t); never more than t."""
    e, t = case["experts"], case.get("tokens", case.get("m"))
    return min(t, e * (1 - (1 - 1 / e) ** t)) if e > 1 else 1.0


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "quantise":
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": n * (size[case["dtype"]] + (2 if case["transposed"] else 1)), "flops": 3 * n}
    if op == "fp8":
        m, n, k = case["m"], case["n"], case["k"]
        used = _touched(case) if case["experts"] else 1
        return {"bytes": m * k + used * n * k + m * n * size[case["out"]], "flops": 2.0 * m * n * k}
    t, n, k, z = case["tokens"], case["n"], case["k"], size[case["dtype"]]
    flops = 2.0 * t * n * k
    if op == "weight_grad":
        return {"bytes": t * (n + k) * z + case["experts"] * n * k * size[case["out"]], "flops": flops}
    return {"bytes": t * (n + k) * z + _touched(case) * n * k * z, "flops": flops}


def _grid_of(v, fmt):
    """float64 values rounded to the 8-bit format's nearest value, ties to even."""
    bits, low = (3, -6) if fmt == "e4m3" else (2, -14)
    exp = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** (low - 8)))).clamp_min(low)
    step = torch.exp2(exp - bits)
    return torch.round(v / step) * step


def _exact_blocks(x, br, fmt):
    """(values on the 8-bit grid, scale) of a float64 matrix, block by block."""
    r, c = x.shape
    rb, cb = -(-r // br), -(-c // BLOCK)
    ri = torch.arange(r, device=x.device) // br
    ci = torch.arange(c, device=x.device) // BLOCK
    col_max = torch.zeros(r, cb, dtype=x.dtype, device=x.device).index_reduce_(1, ci, x.abs(), "amax")
    amax = torch.zeros(rb, cb, dtype=x.dtype, device=x.device).index_reduce_(0, ri, col_max, "amax")
    scale = (amax / (448.0 if fmt == "e4m3" else 57344.0)).clamp_min(SCALE_MIN)
    return _grid_of(x / scale[ri][:, ci], fmt), scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantise":
        x = s["x"].double()
        mats = list(x) if x.dim() == 3 else [x]
        got = [_exact_blocks(v, case["block_rows"], case["fmt"]) for v in mats]
        outs = [[g[i] for g in got] for i in range(2)]
        if case["transposed"]:
            got = [_exact_blocks(v.T.contiguous(), case["block_rows"], case["fmt"]) for v in mats]
            outs += [[g[i] for g in got] for i in range(2)]
        return [torch.stack(o) if x.dim() == 3 else o[0] for o in outs]
    if op == "fp8":
        def wide(q, scale, br):
            rows = torch.arange(q.shape[0], device=q.device) // br
            cols = torch.arange(q.shape[1], device=q.device) // BLOCK
            return q.double() * scale.double()[rows][:, cols]
        a = wide(s["a"], s["a_scale"], 1)
        if not case["experts"]:
            return torch.mm(a, wide(s["b"], s["b_scale"], case["b_rows"]).t().contiguous())
        y = torch.zeros(case["m"], case["n"], dtype=torch.float64, device=DEV)
        for e in range(case["experts"]):
            lo, hi = s["bounds"][e], s["bounds"][e + 1]
            if hi > lo:
                y[lo:hi] = torch.mm(a[lo:hi], wide(s["b"][e], s["b_scale"][e], case["b_rows"]).t().contiguous())
        return y
    y = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for e in range(case["experts"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if hi == lo:
            continue
        if op == "forward":
            y[lo:hi] = torch.mm(s["x"][lo:hi].double(), s["w"][e].double().t().contiguous())
        elif op == "input_grad":
            y[lo:hi] = torch.mm(s["dy"][lo:hi].double(), s["w"][e].double())
        else:
            y[e] = torch.mm(s["dy"][lo:hi].double().t().contiguous(), s["x"][lo:hi].double())
    return y
