"""The measured cases of the 8-bit operators around the optimizer's step and
the expert layers: the AdamW step with its states in 8 bits, the quantisation
of rows to 8-bit integers (of activations, with or without the gated activation
before it, and of weights by output channel), the matrix product of such
operands, and a whole expert layer for a few tokens on bf16 or 8-bit weights.

``listed()`` names the cases, ``draw(rng)`` gives more of the same ranges,
``prepare(case, seed)`` makes what a training or serving program holds before
the call, ``run(state)`` makes one pass: with ``own`` false in plain torch
operations, with ``own`` true through the library.  ``exact`` computes the
same outputs in float64.
"""
import math

import torch

own = False

BLOCK = 128                    # values per scale of an optimizer state
E4M3_MAX, I8_MAX = 448.0, 127.0
SCALE_MIN = 2.0 ** -126        # smallest scale (of values that are all zero)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
DEV = "cuda"


def listed():
    return [
        # training, the norm weights of a small model: launches are all there is
        dict(name="adamw8 norms", op="adamw8", matrices=0, rows=0, cols=2048, vectors=9, dtype="f32", grad="f32",
             packed=False),
        # training, the embedding of a large vocabulary and a model's norm weights: HBM is the bound
        dict(name="adamw8 embedding", op="adamw8", matrices=1, rows=128256, cols=2048, vectors=57, dtype="bf16",
             grad="bf16", packed=False),
        # training in single precision, odd matrices one behind the other in a
        # flat buffer, so that most begin at any address
        dict(name="adamw8 odd", op="adamw8", matrices=5, rows=1001, cols=1543, vectors=40, dtype="f32", grad="bf16",
             packed=True),
        # prefill: the input of a projection
        dict(name="rows activations", op="rows", rows=8192, cols=14336, glu=False, dtype="bf16"),
        # prefill: gate and up as one product left them, the input of the down projection
        dict(name="rows gated", op="rows", rows=8191, cols=4096, glu=True, dtype="bf16"),
        # serving, seven sequences through one projection: the weights are read once
        dict(name="int8 decode", op="int8", m=7, n=14336, k=4096, experts=0, out="bf16", skew=0.0),
        # prefill of one projection: the matrix cores are the bound
        dict(name="int8 prefill", op="int8", m=8192, n=14336, k=4096, experts=0, out="bf16", skew=0.0),
        # prefill of an expert layer
        dict(name="int8 experts", op="int8", m=8192, n=4096, k=2048, experts=16, out="bf16", skew=1.0),
        # odd sizes, single precision results
        dict(name="int8 odd", op="int8", m=1001, n=515, k=1003, experts=0, out="f32", skew=0.0),
        # serving one sequence through wide experts
        dict(name="layer one token", op="layer", tokens=1, experts=8, top_k=2, n=14336, k=4096, weights="bf16"),
        # serving a batch through many narrow experts with 8-bit weights
        dict(name="layer batch int8", op="layer", tokens=32, experts=128, top_k=8, n=1024, k=2048, weights="int8"),
        # a small odd layer: launch latency counts
        dict(name="layer odd", op="layer", tokens=5, experts=16, top_k=3, n=515, k=1000, weights="bf16"),
    ]


MAX_STATES = 128256 * 2048                 # elements of the largest listed optimizer call
MAX_ROWS = 8192 * 14336                    # of the largest listed tensor of rows
MAX_FLOPS = 2.0 * 8192 * 14336 * 4096      # the largest listed product
MAX_WEIGHTS = 3 * 8 * 14336 * 4096         # of the largest listed expert layer


def _size(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A layer's width, even over its logarithm: most are multiples of 128 or
    of 16, one in five is any number."""
    v, kind = _size(rng, lo, hi), rng.random()
    unit = 128 if kind < 0.5 and v >= 128 else 16 if kind < 0.8 and v >= 16 else 1
    return v // unit * unit


def draw(rng):
    while True:
        op = rng.choice(["adamw8", "rows", "int8", "int8", "layer"])
        if op == "adamw8":
            c = dict(op=op, matrices=rng.choice([0, 1, 1, 3, 12]), rows=_size(rng, 1, 128256),
                     cols=_width(rng, 1, 14336), vectors=rng.choice([0, 1, 6, 57]),
                     dtype=rng.choice(["bf16", "bf16", "f32"]), grad=rng.choice(["bf16", "bf16", "f32"]), packed=rng.random() < 0.3)
            c["rows"] = c["rows"] if c["matrices"] else 0
            if 1 <= c["cols"] * (c["matrices"] * c["rows"] + c["vectors"]) <= MAX_STATES // 2:
                return c
        elif op == "rows":
            c = dict(op=op, rows=_size(rng, 1, 14336), cols=_width(rng, 16, 14336), glu=rng.random() < 0.4,
                     dtype=rng.choice(["bf16", "bf16", "f32"]))
            if 2 ** 12 <= c["rows"] * c["cols"] * (2 if c["glu"] else 1) <= MAX_ROWS // 2:
                return c
        elif op == "int8":
            e = rng.choice([0, 0, 4, 16, 61])
            c = dict(op=op, m=_size(rng, 1, 8192), n=_width(rng, 16, 14336), k=_width(rng, 32, 14336), experts=e,
                     out=rng.choice(["bf16", "bf16", "f32"]), skew=rng.choice([0.5, 1.0, 2.0]) if e else 0.0)
            if 2.0 * c["m"] * c["n"] * c["k"] <= MAX_FLOPS and max(1, e) * c["n"] * c["k"] <= MAX_WEIGHTS // 3:
                return c
        else:
            e = rng.choice([4, 8, 16, 64, 128, 256])
            c = dict(op=op, tokens=_size(rng, 1, 64), experts=e, top_k=rng.choice([1, 2, 2, 4, 6, 8]),
                     n=_width(rng, 64, 14336), k=_width(rng, 128, 8192), weights=rng.choice(["bf16", "int8"]))
            if c["top_k"] <= e and 3 * e * c["n"] * c["k"] <= MAX_WEIGHTS:
                return c


def _normal(gen, shape, std, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).mul_(std).to(dtype)


def _outliers(x, gen):
    """A few columns thirty times as large, as activations have them."""
    cols = torch.randint(0, x.shape[-1], (max(1, x.shape[-1] // 256),), generator=gen, device=DEV)
    x[..., cols] *= 30
    return x


def _to_rows(x):
    """Values (..., c) -> (8-bit integers, fp32 scale per row), in fp32:
    scale = amax / 127, x * (1 / scale) rounded to nearest even."""
    scale = (x.float().abs().amax(-1) / I8_MAX).clamp_min(SCALE_MIN)
    return torch.round(x.float() * (1.0 / scale)[..., None]).to(torch.int8), scale


def _to_state(x, random=None):
    """A flat fp32 tensor -> (e4m3 values, fp32 scale per 128), in fp32:
    scale = amax / 448, x * (1 / scale) rounded to nearest even, or, with
    random numbers in [0, 1) for values that are not negative, up where the
    part cut off and the random number are 1 or more together."""
    n = x.numel()
    xb = torch.nn.functional.pad(x, (0, -n % BLOCK)).view(-1, BLOCK)
    scale = (xb.abs().amax(1) / E4M3_MAX).clamp_min(SCALE_MIN)
    y = (xb * (1.0 / scale)[:, None]).view(-1)[:n]
    if random is not None:
        y = y.clamp_max(E4M3_MAX)
        # the bits of the power of two of y, no less than the smallest normal number's
        exp = (y.view(torch.int32) & 0x7f800000).clamp_min(121 << 23)
        step, steps = (exp - (3 << 23)).view(torch.float32), ((257 << 23) - exp.long()).int().view(torch.float32)
        y = torch.floor(y * steps + random) * step
    return y.to(torch.float8_e4m3fn), scale


def _mix(x):
    """A 32-bit hash (the finaliser of MurmurHash3, of x + 0x9e3779b9) of a number or a tensor of int64."""
    x = (x + 0x9e3779b9) & 0xffffffff
    x = ((x ^ (x >> 16)) * 0x85ebca6b) & 0xffffffff
    x = ((x ^ (x >> 13)) * 0xc2b2ae35) & 0xffffffff
    return x ^ (x >> 16)


def _random(seed, step, tensor, n):
    """The random numbers of a step for the n elements of a tensor: 16 bits
    each, two from one hash of the call's seed, the step, the tensor's place in
    the call and the pair's place in the tensor."""
    key = _mix(_mix(_mix(seed) + step) + tensor)
    pair = torch.arange((n + 1) // 2, device=DEV)
    word = _mix(_mix(key + (pair >> 12)) + (pair & 4095))
    return torch.stack((word & 0xffff, word >> 16), 1).view(-1)[:n]


def _of_state(q, scale):
    """The fp32 values that an 8-bit state stands for."""
    return q.float() * scale.repeat_interleave(BLOCK)[:q.numel()]


def _counts(g, experts, tokens, skew):
    """Tokens per expert: a routing with popular and unpopular experts (the
    popularity's logarithm is normal with deviation `skew`)."""
    p = torch.exp(skew * torch.randn(experts, generator=g, dtype=torch.float64))
    return torch.bincount(torch.multinomial(p, tokens, replacement=True, generator=g), minlength=experts)


GROUPS = [dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01),     # matrices
          dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0)]      # vectors


def _prepare_adamw8(case, gen):
    """The tensors are pieces of flat buffers, as a trainer's buckets hold
    them: at multiples of 128 elements, or one right behind the other."""
    sizes = [case["rows"] * case["cols"]] * case["matrices"] + [case["cols"]] * case["vectors"]
    at, sat, n, ns = [], [], 0, 0
    for size in sizes:
        at.append(n)
        sat.append(ns)
        n += size if case["packed"] else -(-size // BLOCK) * BLOCK
        ns += -(-size // BLOCK)
    g = _normal(gen, (n,), 1e-3)
    # gradients of rare and of frequent words differ by orders of magnitude
    g[:n // 64 * 64].view(n // 64, 64).mul_(torch.exp(1.5 * _normal(gen, (n // 64, 1), 1.0)))
    root = g.abs().mul_(0.5 + torch.rand(n, generator=gen, device=DEV))
    avg = g * 0.3 + root * _normal(gen, (n,), 0.2)
    s = dict(step=100, seed=int(torch.randint(2 ** 31, (1,), generator=gen, device=DEV)))
    s["p"] = _normal(gen, (n,), 0.02, DT[case["dtype"]])
    s["g"] = (g + 1e-4 * _normal(gen, (n,), 1.0)).to(DT[case["grad"]])
    s["avg"] = torch.zeros(n, dtype=torch.float8_e4m3fn, device=DEV)
    s["root"] = torch.zeros(n, dtype=torch.float8_e4m3fn, device=DEV)
    s["avg_scale"] = torch.zeros(ns, device=DEV)
    s["root_scale"] = torch.zeros(ns, device=DEV)
    for a, b, size in zip(at, sat, sizes):
        for v, name in ((avg, "avg"), (root, "root")):
            q, scale = _to_state(v[a:a + size])
            s[name][a:a + size] = q
            s[name + "_scale"][b:b + scale.numel()] = scale
    for name in ("p", "g", "avg", "root"):
        s[name + "s"] = [s[name][a:a + size] for a, size in zip(at, sizes)]
    for name in ("avg_scale", "root_scale"):
        s[name + "s"] = [s[name][b:b + -(-size // BLOCK)] for b, size in zip(sat, sizes)]
    s["group_index"] = [0] * case["matrices"] + [1] * case["vectors"]
    return s


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    op = case["op"]
    s = dict(op=op)
    if op == "adamw8":
        s.update(_prepare_adamw8(case, gen))
    elif op == "rows":
        r, c, glu = case["rows"], case["cols"], case["glu"]
        x = _outliers(_normal(gen, (r, 2 * c if glu else c), 0.5), gen)
        s.update(x=x.to(DT[case["dtype"]]), glu=glu)
        s["q"] = torch.empty(r, c, dtype=torch.int8, device=DEV)
        s["scale"] = torch.empty(r, dtype=torch.float32, device=DEV)
        if glu:
            s["values"] = torch.empty(r, c, dtype=torch.bfloat16, device=DEV)
    elif op == "int8":
        m, n, k, e = case["m"], case["n"], case["k"], case["experts"]
        s["a"], s["a_scale"] = _to_rows(_outliers(_normal(gen, (m, k), 0.5), gen))
        s["b"], s["b_scale"] = _to_rows(_normal(gen, (e, n, k) if e else (n, k), 0.02))
        s["c"] = torch.zeros(m, n, dtype=DT[case["out"]], device=DEV)
        s["bounds"] = s["offsets"] = None
        if e:
            s["bounds"] = [0] + torch.cumsum(_counts(host, e, m, case["skew"]), 0).tolist()
            s["offsets"] = torch.tensor(s["bounds"], dtype=torch.int32, device=DEV)
    else:
        t, e, n, k = case["tokens"], case["experts"], case["n"], case["k"]
        s["x"] = _outliers(_normal(gen, (t, k), 0.5), gen).to(torch.bfloat16)
        popular = torch.exp(torch.randn(e, generator=host)).expand(t, e)
        ids = torch.multinomial(popular, case["top_k"], generator=host)
        s["ids"] = ids.to(torch.int32).to(DEV)
        s["touched"] = sorted(set(ids.flatten().tolist()))
        s["gates"] = torch.softmax(torch.randn(t, case["top_k"], generator=host), 1).to(DEV)
        s["w_in"], s["w_out"] = (_normal(gen, shape, 0.02, torch.bfloat16) for shape in ((e, 2 * n, k), (e, k, n)))
        s["in_scale"] = s["out_scale"] = None
        if case["weights"] == "int8":
            s["w_in"], s["in_scale"] = _to_rows(s["w_in"])
            s["w_out"], s["out_scale"] = _to_rows(s["w_out"])
        s["y"] = torch.zeros(t, k, dtype=torch.bfloat16, device=DEV)
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"adamw8": _adamw8, "rows": _rows, "int8": _int8, "layer": _layer}[s["op"]](s)


def _adamw8(s):
    """Every rounding in fp32, in this order; the second moment is held by its
    root, which is rounded at random: one step moves it by a small part of
    what 8 bits can tell apart, and rounded to nearest it would never move."""
    s["step"] += 1
    every = zip(s["ps"], s["gs"], s["avgs"], s["avg_scales"], s["roots"], s["root_scales"])
    for i, (p, g, avg, avg_scale, root, root_scale) in enumerate(every):
        h = GROUPS[s["group_index"][i]]
        b1, b2 = h["betas"]
        g = g.float()
        m = b1 * _of_state(avg, avg_scale) + (1 - b1) * g
        r = _of_state(root, root_scale)
        r = torch.sqrt(b2 * (r * r) + (1 - b2) * (g * g))
        denom = r * (1 / math.sqrt(1 - b2 ** s["step"])) + h["eps"]
        w = p.float() * (1 - h["lr"] * h["weight_decay"]) - (h["lr"] / (1 - b1 ** s["step"])) * (m / denom)
        p.copy_(w.to(p.dtype))
        random = _random(s["seed"], s["step"], i, p.numel()).float() * 2.0 ** -16
        for v, q, scale, u in ((m, avg, avg_scale, None), (r, root, root_scale, random)):
            new, new_scale = _to_state(v, u)
            q.copy_(new)
            scale.copy_(new_scale)
    return _states(s)


def _states(s):
    return {k: s[k] for k in ("p", "avg", "avg_scale", "root", "root_scale")}


def _rows(s):
    x = s["x"].float()
    if not s["glu"]:
        return _to_rows(x)
    gate, up = x.chunk(2, 1)
    q, scale = _to_rows(gate / (1 + torch.exp(-gate)) * up)
    # the integers as the values that they stand for
    return (q.float() * scale[:, None]).to(torch.bfloat16), scale


def _int8(s):
    a, bounds = s["a"].float(), s["bounds"]
    if bounds is None:
        c = a @ s["b"].float().T * s["a_scale"][:, None] * s["b_scale"]
        return c.to(s["c"].dtype)
    parts = [a[lo:hi] @ s["b"][e].float().T * s["a_scale"][lo:hi, None] * s["b_scale"][e]
             for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])) if hi > lo]
    return torch.cat(parts).to(s["c"].dtype)


def _layer(s):
    x, y = s["x"].float(), 0
    for e in s["touched"]:
        w_in, w_out = s["w_in"][e].float(), s["w_out"][e].float()
        if s["in_scale"] is not None:
            w_in, w_out = w_in * s["in_scale"][e][:, None], w_out * s["out_scale"][e][:, None]
        gate, up = (x @ w_in.T).chunk(2, 1)
        share = (s["gates"] * (s["ids"] == e)).sum(1, keepdim=True)
        y = y + share * ((gate / (1 + torch.exp(-gate)) * up) @ w_out.T)
    return y.to(torch.bfloat16)


def _run_own(s):
    import matrix_optimizer_step_owned_amd as dm
    op = s["op"]
    if op == "adamw8":
        s["step"] += 1
        dm.dmuon_adamw_step_quantized(s["ps"], s["gs"], s["avgs"], s["avg_scales"], s["roots"], s["root_scales"],
                                      groups=[dict(h, step=s["step"]) for h in GROUPS], group_index=s["group_index"],
                                      seed=s["seed"])
        return _states(s)
    if op == "rows":
        q, scale = dm.dmuon_quantize_rows(s["x"], activation="swiglu" if s["glu"] else None, q=s["q"], scale=s["scale"])
        return (dm.dmuon_dequantize_rows(q, scale, out=s["values"]) if s["glu"] else q), scale
    if op == "int8":
        return dm.dmuon_row_matmul(s["a"], s["a_scale"], s["b"], s["b_scale"], offsets=s["offsets"], out=s["c"])
    return dm.dmuon_expert_layer(s["x"], s["ids"], s["gates"], s["w_in"], s["w_out"], in_scale=s["in_scale"],
                                 out_scale=s["out_scale"], out=s["y"])


def _touched(e, picks):
    """Experts that get a row, as expected over routings that know no
    favourites; never more than there are rows."""
    return min(picks, e * (1 - (1 - 1 / e) ** picks)) if e > 1 else 1.0


def work(case):
    size = {"bf16": 2, "f32": 4}
    op = case["op"]
    if op == "adamw8":
        # p read and written, the gradient read, two states and their scales read and written
        n = case["cols"] * (case["matrices"] * case["rows"] + case["vectors"])
        return {"bytes": n * (2 * size[case["dtype"]] + size[case["grad"]] + 4 * (1 + 4 / BLOCK)), "flops": 20 * n}
    if op == "rows":
        n = case["rows"] * case["cols"]
        if not case["glu"]:
            return {"bytes": n * (size[case["dtype"]] + 1) + 4 * case["rows"], "flops": 3 * n}
        # the integers are read again for the values that they stand for
        return {"bytes": n * (2 * size[case["dtype"]] + 1 + 1 + 2) + 4 * case["rows"], "flops": 9 * n}
    if op == "int8":
        m, n, k, e = case["m"], case["n"], case["k"], case["experts"]
        used = _touched(e, m) if e else 1
        return {"bytes": m * (k + 4) + used * n * (k + 4) + m * n * size[case["out"]], "flops": 2.0 * m * n * k}
    t, n, k, e = case["tokens"], case["n"], case["k"], case["experts"]
    picks = t * case["top_k"]
    used = _touched(e, picks)
    weight = 2 if case["weights"] == "bf16" else 1
    return {"bytes": used * 3 * n * k * weight + t * k * 4 + picks * 8, "flops": 6.0 * picks * n * k}


def _grid_e4m3(v, random=None):
    """float64 values rounded to the nearest e4m3 value, ties to even, or at random."""
    exp = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -14))).clamp_min(-6)
    step = torch.exp2(exp - 3)
    return (torch.round(v / step) if random is None else torch.floor(v / step + random)) * step


def _exact_adamw8(s):
    out = {k: s[k].double().clone() for k in ("p", "avg", "avg_scale", "root", "root_scale")}
    t = s["step"] + 1
    for i, k in enumerate(s["group_index"]):
        a, n = s["ps"][i].storage_offset(), s["ps"][i].numel()
        b, nb = s["avg_scales"][i].storage_offset(), s["avg_scales"][i].numel()
        blk = torch.arange(n, device=DEV) // BLOCK
        lr, (b1, b2), eps, wd = (GROUPS[k][w] for w in ("lr", "betas", "eps", "weight_decay"))
        g = s["gs"][i].double()
        m = out["avg"][a:a + n] * out["avg_scale"][b:b + nb][blk]
        m = m + (1 - b1) * (g - m)
        v = (out["root"][a:a + n] * out["root_scale"][b:b + nb][blk]) ** 2
        v = v + (1 - b2) * (g * g - v)
        p = out["p"][a:a + n]
        p -= lr * wd * p + lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
        random = _random(s["seed"], t, i, n).double() / 65536
        for name, x, u in (("avg", m, None), ("root", v.sqrt(), random)):
            scale = torch.zeros(nb, dtype=torch.float64, device=DEV).index_reduce_(0, blk, x.abs(), "amax") / E4M3_MAX
            scale = scale.clamp_min(SCALE_MIN)
            out[name + "_scale"][b:b + nb] = scale
            out[name][a:a + n] = _grid_e4m3((x / scale[blk]).clamp_max(E4M3_MAX), u)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "adamw8":
        return _exact_adamw8(s)
    if op == "rows":
        x = s["x"].double()
        if case["glu"]:
            x = torch.nn.functional.silu(x[:, :case["cols"]]) * x[:, case["cols"]:]
        scale = (x.abs().max(1).values / 127).clamp_min(SCALE_MIN)
        q = torch.round(x / scale.unsqueeze(1))
        return (q * scale.unsqueeze(1) if case["glu"] else q.to(torch.int8)), scale
    if op == "int8":
        y = torch.empty(case["m"], case["n"], dtype=torch.float64, device=DEV)
        spans = [(0, case["m"], s["b"], s["b_scale"])]
        if case["experts"]:
            spans = [(s["bounds"][e], s["bounds"][e + 1], s["b"][e], s["b_scale"][e]) for e in range(case["experts"])]
        for lo, hi, b, scale in spans:
            w = b.double().mul_(scale.double().unsqueeze(1)).t().contiguous()
            y[lo:hi] = torch.mm(s["a"][lo:hi].double() * s["a_scale"][lo:hi].double().unsqueeze(1), w)
        return y
    y = torch.zeros(case["tokens"], case["k"], dtype=torch.float64, device=DEV)
    for e in s["touched"]:
        w = [s["w_in"][e].double(), s["w_out"][e].double()]
        if case["weights"] == "int8":
            w = [v * scale[e].double().unsqueeze(1) for v, scale in zip(w, (s["in_scale"], s["out_scale"]))]
        token, pick = torch.nonzero(s["ids"] == e, as_tuple=True)
        h = torch.mm(s["x"].double()[token], w[0].t().contiguous())
        h = torch.nn.functional.silu(h[:, :case["n"]]) * h[:, case["n"]:]
        y.index_add_(0, token, torch.mm(h * s["gates"].double()[token, pick].unsqueeze(1), w[1].t().contiguous()))
    return y
