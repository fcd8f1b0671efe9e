"""Refusals of the AdamW step with 8-bit states, of the 8-bit integer rows and their product and of
the expert layer (CPU): every check runs before any launch, so fake addresses are never read."""
import ctypes

import pytest

BASE, M = 1 << 30, 1 << 20


@pytest.fixture(scope="module")
def dm():
    import matrix_optimizer_step_owned_amd as dm
    return dm


def test_struct_sizes(dm):
    assert ctypes.sizeof(dm.dmuon_adamw_quantized_t) == dm._ADAMW8_TENSOR.size == 72
    assert ctypes.sizeof(dm.dmuon_rows_t) == 32
    assert ctypes.sizeof(dm.dmuon_row_product_t) == 72
    assert ctypes.sizeof(dm.dmuon_expert_layer_t) == 88


def fill(d, values, kw):
    values.update(kw)
    for k, x in values.items():
        setattr(d, k, x)
    return d


def adam(dm, base=BASE, **kw):
    return fill(dm.dmuon_adamw_quantized_t(), dict(
        numel=1000, param=base, grad=base + M, exp_avg=base + 2 * M, exp_avg_scale=base + 3 * M, root=base + 4 * M,
        root_scale=base + 5 * M, param_dtype=1, grad_dtype=1, group=0), kw)


def group(dm, **kw):
    return fill(dm.dmuon_adamw_group_t(), dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1), kw)


def test_adamw_refusals(dm):
    def call(ts, gs=None, n=None):
        gs = [group(dm)] if gs is None else gs
        ta = (dm.dmuon_adamw_quantized_t * max(len(ts), 1))(*ts)
        ga = (dm.dmuon_adamw_group_t * max(len(gs), 1))(*gs)
        return dm._lib.dmuon_adamw_step_quantized(ta, len(ts) if n is None else n, ga, len(gs), 0, None)

    bad = dm.DMUON_ERR_INVALID_ARG
    assert call([], n=-1) == bad
    assert call([]) == dm.DMUON_OK
    assert dm._lib.dmuon_adamw_step_quantized(None, 1, None, 1, 0, None) == bad
    assert call([adam(dm)], gs=[]) == bad
    for kw in (dict(lr=float("nan")), dict(weight_decay=float("inf")), dict(eps=-1e-8), dict(eps=float("nan")),
               dict(beta1=1.0), dict(beta2=-0.1), dict(beta1=float("nan")), dict(step=0)):
        assert call([adam(dm)], [group(dm, **kw)]) == bad, kw
        assert "groups[0]" in dm.dmuon_last_error()
    for kw in (dict(numel=-1), dict(numel=(1 << 42) + 1), dict(group=1), dict(group=-1), dict(param=None),
               dict(exp_avg=None), dict(exp_avg_scale=None), dict(root=None), dict(root_scale=None),
               dict(param=BASE + 1), dict(grad=BASE + M + 1), dict(exp_avg_scale=BASE + 3 * M + 2),
               dict(root_scale=BASE + 5 * M + 1)):
        assert call([adam(dm), adam(dm, BASE + 9 * M, **kw)]) == bad, kw
        assert "tensors[1]" in dm.dmuon_last_error()
    for kw in (dict(param_dtype=2), dict(grad_dtype=4)):
        assert call([adam(dm, **kw)]) == dm.DMUON_ERR_UNSUPPORTED, kw
    for kw in (dict(root=BASE + 2 * M), dict(grad=BASE + 10), dict(root_scale=BASE + 3 * M + 28)):
        assert call([adam(dm, **kw)]) == dm.DMUON_ERR_ALIASING, kw
    assert call([adam(dm), adam(dm)]) == dm.DMUON_ERR_ALIASING
    assert "tensors[" in dm.dmuon_last_error() and "overlaps" in dm.dmuon_last_error()
    # nothing to do: no gradient, no elements
    assert call([adam(dm, grad=None), adam(dm, numel=0)]) == dm.DMUON_OK


def test_rows_refusals(dm):
    x, q, s = BASE, BASE + M, BASE + 2 * M
    bad = dm.DMUON_ERR_INVALID_ARG

    def rows(**kw):
        return fill(dm.dmuon_rows_t(), dict(rows=100, cols=300, ldx=300, x_dtype=1, activation=0), kw)

    quant = lambda d, x=x, q=q, s=s: dm._lib.dmuon_quantize_rows(d, x, q, s, None)
    deq = lambda d, x=x, q=q, s=s: dm._lib.dmuon_dequantize_rows(d, q, s, x, None)
    for f in (quant, deq):
        assert f(None) == bad
        for kw in (dict(rows=-1), dict(rows=(1 << 30) + 1), dict(cols=0), dict(cols=(1 << 22) + 1, ldx=1 << 23),
                   dict(ldx=299), dict(ldx=(1 << 23) + 1), dict(activation=2), dict(activation=1, ldx=599)):
            assert f(rows(**kw)) == bad, kw
        for dt in (2, 3, 4, -1):
            assert f(rows(x_dtype=dt)) == dm.DMUON_ERR_UNSUPPORTED
        for kw in (dict(x=None), dict(q=None), dict(s=None), dict(x=x + 1), dict(s=s + 2)):
            assert f(rows(), **kw) == bad, kw
        assert f(rows(), q=x) == dm.DMUON_ERR_ALIASING
        assert f(rows(rows=0), x=None) == dm.DMUON_OK
    assert quant(rows(), s=q) == dm.DMUON_ERR_ALIASING
    assert quant(rows(activation=1, ldx=600), q=x + 2 * 550) == dm.DMUON_ERR_ALIASING     # in the half that is up
    assert deq(rows(activation=1, ldx=600)) == bad


def test_matmul_refusals(dm):
    a, sa, b, sb, c, off = (BASE + i * M for i in range(6))
    bad = dm.DMUON_ERR_INVALID_ARG

    def product(**kw):
        return fill(dm.dmuon_row_product_t(), dict(m=10, n=200, k=300, lda=300, ldb=300, ldc=200, b_stride=0, experts=0,
                                                   out_dtype=1, accumulate=0), kw)

    def call(d, a=a, sa=sa, b=b, sb=sb, off=None, c=c):
        return dm._lib.dmuon_row_matmul(d, a, sa, b, sb, off, c, None)

    assert call(None) == bad
    for kw in (dict(m=-1), dict(m=(1 << 30) + 1), dict(n=0), dict(n=(1 << 22) + 1, ldc=1 << 23), dict(k=0),
               dict(k=131072, lda=131072, ldb=131072), dict(lda=299), dict(ldb=299), dict(ldc=199), dict(experts=-1),
               dict(experts=65537), dict(accumulate=2), dict(experts=2)):
        assert call(product(**kw)) == bad, kw
    assert call(product(), off=off) == bad
    assert call(product(experts=2, b_stride=200 * 300 - 1), off=off) == bad
    assert call(product(out_dtype=4)) == dm.DMUON_ERR_UNSUPPORTED
    for kw in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None), dict(c=c + 1), dict(sa=sa + 1),
               dict(sb=sb + 2)):
        assert call(product(), **kw) == bad, kw
    for other in (a, b, sa, sb):
        assert call(product(), c=other) == dm.DMUON_ERR_ALIASING
    assert call(product(experts=2, b_stride=60000), off=c + 400, b=BASE + 9 * M) == dm.DMUON_ERR_ALIASING
    assert call(product(m=0), a=None) == dm.DMUON_OK
    assert call(product(m=1 << 30, n=1 << 22, ldc=1 << 22), sa=1 << 40, b=1 << 50, c=1 << 55) == dm.DMUON_ERR_UNSUPPORTED


def test_layer_refusals(dm):
    x, ids, gates, w_in, w_out, y, ws, si, so = (BASE + i * (8 * M) for i in range(9))
    bad = dm.DMUON_ERR_INVALID_ARG

    def layer(**kw):
        return fill(dm.dmuon_expert_layer_t(), dict(
            tokens=10, n=48, k=64, ldx=64, ldy=64, ld_in=64, ld_out=48, in_stride=96 * 64, out_stride=64 * 48, experts=8,
            top_k=2, weight_dtype=1), kw)

    def call(d, x=x, ids=ids, gates=gates, w_in=w_in, si=None, w_out=w_out, so=None, y=y, ws=ws, wsb=1 << 22):
        return dm._lib.dmuon_expert_layer(d, x, ids, gates, w_in, si, w_out, so, y, ws, wsb, None)

    need = dm._lib.dmuon_expert_layer_workspace_size
    assert need(layer()) >= 10 * 2 * 48 * 4 and need(layer(n=45)) == need(layer())
    assert need(None) == 0 and need(layer(tokens=0)) == 0 and need(layer(tokens=65)) == 0
    assert need(layer(k=0)) == 0
    assert call(None) == bad
    for kw in (dict(tokens=-1), dict(tokens=65), dict(n=0), dict(k=0), dict(experts=0), dict(experts=4097), dict(top_k=0),
               dict(top_k=65), dict(ldx=63), dict(ldy=63), dict(ld_in=63), dict(ld_out=47), dict(ldx=(1 << 22) + 1),
               dict(in_stride=96 * 64 - 1), dict(out_stride=64 * 48 - 1), dict(in_stride=1 << 45)):
        assert call(layer(**kw)) == bad, kw
    for dt in (0, 2, 3):
        assert call(layer(weight_dtype=dt)) == dm.DMUON_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(ids=None), dict(gates=None), dict(w_in=None), dict(w_out=None), dict(y=None),
               dict(x=x + 1), dict(y=y + 1), dict(w_in=w_in + 1), dict(ids=ids + 2), dict(gates=gates + 1), dict(ws=ws + 8),
               dict(si=si), dict(so=so)):
        assert call(layer(), **kw) == bad, kw
    assert call(layer(weight_dtype=4), si=si) == bad
    assert call(layer(weight_dtype=4), si=si, so=so + 2) == bad
    assert call(layer(), ws=None) == dm.DMUON_ERR_WORKSPACE
    assert call(layer(), wsb=need(layer()) - 1) == dm.DMUON_ERR_WORKSPACE
    for kw in (dict(y=x), dict(y=ids), dict(y=w_in + 2 * 96 * 64 * 7), dict(ws=w_out), dict(ws=y), dict(ws=gates)):
        assert call(layer(), **kw) == dm.DMUON_ERR_ALIASING, kw
    assert call(layer(weight_dtype=4), si=si, so=y) == dm.DMUON_ERR_ALIASING
    assert call(layer(tokens=0), x=None, ws=None) == dm.DMUON_OK
    big = dict(tokens=64, top_k=64, experts=4096, n=1 << 22, ld_out=1 << 22, in_stride=1 << 40, out_stride=1 << 40)
    assert call(layer(**big), w_in=1 << 60, w_out=1 << 61, wsb=1 << 62, ws=1 << 57) == dm.DMUON_ERR_UNSUPPORTED


def test_binding_refusals(dm):
    import torch
    bf, f8, i8 = torch.bfloat16, torch.float8_e4m3fn, torch.int8
    p, g, s = torch.zeros(200), torch.zeros(200), torch.zeros(2)
    m = torch.zeros(200, dtype=f8)
    with pytest.raises(ValueError):
        dm.dmuon_adamw_step_quantized([p], [g], [m], [s], [m], [], step=1)
    with pytest.raises(ValueError):
        dm.dmuon_adamw_step_quantized([p], [g], [m], [s], [m], [s], step=1, seed=-1)
    with pytest.raises(ValueError):
        dm.dmuon_adamw_step_quantized([p], [g], [m], [s], [m], [s], groups=[dict(step=1)])
    with pytest.raises(ValueError):
        dm.dmuon_adamw_step_quantized([p], [g], [m], [s], [m], [s], step=1)        # not on a GPU
    dm.dmuon_adamw_step_quantized([], [], [], [], [], [], step=1)
    st = dm.dmuon_adamw_quantized_state(torch.zeros(3, 43))
    assert st[0].dtype == f8 and st[0].shape == (3, 43) and st[1].shape == (2,) and st[3].dtype == torch.float32
    x = torch.zeros(4, 6, dtype=bf)
    for bad in (x[0], torch.zeros(2, 4, 6)[:, ::2], x.t()):
        with pytest.raises(ValueError):
            dm.dmuon_quantize_rows(bad)
    with pytest.raises(ValueError):
        dm.dmuon_quantize_rows(x[:, :5], activation="swiglu")
    for none in (x[:, :0], x.view(2, 2, 6)[..., :0].contiguous()):
        for act in (None, "swiglu"):
            with pytest.raises(ValueError, match="columns"):
                dm.dmuon_quantize_rows(none, activation=act)
    with pytest.raises(KeyError):
        dm.dmuon_quantize_rows(x, activation="gelu")
    with pytest.raises(ValueError):
        dm.dmuon_quantize_rows(x)                                                   # not on a GPU
    with pytest.raises(ValueError):
        dm.dmuon_quantize_rows(x.float().requires_grad_())
    q, sc = torch.zeros(4, 8, dtype=i8), torch.ones(4)
    off = torch.zeros(3, dtype=torch.int32)
    for args, kw in (((q, sc[:3], q, sc), {}), ((q, sc, q[:, :7], sc), {}), ((q, sc, q, sc[None]), {}),
                     ((q, sc, q, sc), dict(accumulate=True)), ((q, sc, q[None], sc[None]), dict(offsets=off)),
                     ((q, sc, q, sc), {})):
        with pytest.raises(ValueError):
            dm.dmuon_row_matmul(*args, **kw)
    with pytest.raises(TypeError):
        dm.dmuon_row_matmul(x, sc, x, sc)
    w_in, w_out = torch.zeros(2, 10, 6, dtype=bf), torch.zeros(2, 6, 5, dtype=bf)
    ids, gates = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    for args, kw in (((x, ids, gates, w_in[:, :8], w_out), {}), ((x, ids[:3], gates, w_in, w_out), {}),
                     ((x, ids, gates[:, :1], w_in, w_out), {}), ((x, ids.long(), gates, w_in, w_out), {}),
                     ((x, ids, gates, w_in, w_out[:1]), {}), ((x, ids, gates, w_in, w_out), dict(in_scale=sc)),
                     ((x, ids, gates, w_in.to(i8), w_out.to(i8)), {}), ((x, ids, gates, w_in, w_out), {}),
                     ((x, ids, gates.requires_grad_(), w_in, w_out), {})):
        with pytest.raises(ValueError):
            dm.dmuon_expert_layer(*args, **kw)
    with pytest.raises(TypeError):
        dm.dmuon_expert_layer(x.float(), ids, gates.detach(), w_in, w_out)
    with pytest.raises(TypeError):
        dm.dmuon_expert_layer(x, ids, gates.detach(), w_in, w_out.to(i8))
