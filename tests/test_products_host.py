"""Refusals of the expert products and the 8-bit block operators (CPU): every
check runs before any launch, so fake addresses are never read."""
import ctypes

import pytest

BASE = 1 << 30


@pytest.fixture(scope="module")
def dm():
    import matrix_optimizer_step_owned_amd as dm
    return dm


def test_struct_sizes(dm):
    assert ctypes.sizeof(dm.dmuon_experts_t) == 72
    assert ctypes.sizeof(dm.dmuon_blocks_t) == 56
    assert ctypes.sizeof(dm.dmuon_block_product_t) == 80


def experts(dm, **kw):
    d = dm.dmuon_experts_t()
    v = dict(tokens=10, n=32, k=64, ld_k=64, ld_n=32, ldw=64, w_stride=32 * 64, experts=3, dtype=1, out_dtype=1,
             accumulate=0)
    v.update(kw)
    for k, x in v.items():
        setattr(d, k, x)
    return d


PRODUCTS = ["dmuon_expert_matmul", "dmuon_expert_input_grad", "dmuon_expert_weight_grad"]


@pytest.mark.parametrize("name", PRODUCTS)
def test_expert_refusals(dm, name):
    f = getattr(dm._lib, name)
    a, b, off, c = BASE, BASE + (1 << 20), BASE + (2 << 20), BASE + (3 << 20)

    def call(d, a=a, b=b, off=off, c=c):
        return f(d, a, b, off, c, None)

    bad = dm.DMUON_ERR_INVALID_ARG
    for kw in (dict(tokens=-1), dict(tokens=(1 << 30) + 1), dict(n=0), dict(k=0), dict(n=1 << 23, ld_n=1 << 23),
               dict(experts=0), dict(experts=65537), dict(ld_k=63), dict(ld_n=31), dict(ldw=63),
               dict(ldw=(1 << 22) + 1), dict(w_stride=31 * 64 + 63), dict(w_stride=1 << 45), dict(accumulate=2)):
        assert call(experts(dm, **kw)) == bad, kw
    assert call(None) == bad
    assert call(experts(dm, dtype=2)) == dm.DMUON_ERR_UNSUPPORTED
    for kw in (dict(a=None), dict(b=None), dict(off=None), dict(c=None), dict(a=a + 1), dict(b=b + 1), dict(c=c + 1),
               dict(off=off + 2)):
        assert call(experts(dm), **kw) == bad, kw
    assert call(experts(dm), c=a) == dm.DMUON_ERR_ALIASING
    assert "overlaps" in dm.dmuon_last_error()
    assert call(experts(dm), c=b + 2) == dm.DMUON_ERR_ALIASING
    assert call(experts(dm), c=off) == dm.DMUON_ERR_ALIASING
    big = dict(n=1 << 22, ld_n=1 << 22, k=1 << 22, ld_k=1 << 22, ldw=1 << 22, w_stride=1 << 44, tokens=1 << 20)
    assert call(experts(dm, **big), b=1 << 50, c=1 << 60) == dm.DMUON_ERR_UNSUPPORTED
    if name == "dmuon_expert_weight_grad":
        assert call(experts(dm, dtype=0, out_dtype=1)) == dm.DMUON_ERR_UNSUPPORTED
        assert call(experts(dm, out_dtype=3)) == dm.DMUON_ERR_UNSUPPORTED
        assert call(experts(dm, tokens=0, accumulate=1)) == dm.DMUON_OK
    else:
        assert call(experts(dm, accumulate=1)) == bad
        assert call(experts(dm, tokens=0), a=None, c=None) == dm.DMUON_OK


def blocks(dm, **kw):
    d = dm.dmuon_blocks_t()
    v = dict(batch=1, rows=200, cols=300, ldx=300, x_stride=0, block_rows=1, x_dtype=1, q_dtype=2)
    v.update(kw)
    for k, x in v.items():
        setattr(d, k, x)
    return d


def test_quantize_refusals(dm):
    M = 1 << 20
    x, q, s, qt, st = (BASE + i * M for i in range(5))
    bad = dm.DMUON_ERR_INVALID_ARG

    def quant(d, x=x, q=q, s=s, qt=qt, st=st):
        return dm._lib.dmuon_quantize_blocks(d, x, q, s, qt, st, None)

    def deq(d, x=x, q=q, s=s):
        return dm._lib.dmuon_dequantize_blocks(d, q, s, x, None)

    for f in (quant, deq):
        for kw in (dict(batch=0), dict(batch=65536), dict(rows=-1), dict(cols=0), dict(ldx=299), dict(block_rows=64),
                   dict(rows=(1 << 30) + 1), dict(batch=2, x_stride=100)):
            assert f(blocks(dm, **kw)) == bad, kw
        assert f(None) == bad
        for kw in (dict(x_dtype=2), dict(q_dtype=1), dict(rows=1 << 30, cols=1 << 20, ldx=1 << 20)):
            assert f(blocks(dm, **kw)) == dm.DMUON_ERR_UNSUPPORTED, kw
        assert f(blocks(dm), x=None) == bad
        assert f(blocks(dm), x=x + 1) == bad
        assert f(blocks(dm), s=s + 2) == bad
        assert f(blocks(dm), q=x) == dm.DMUON_ERR_ALIASING
        assert f(blocks(dm, rows=0)) == dm.DMUON_OK
    assert quant(blocks(dm), q=None) == bad
    assert quant(blocks(dm), st=None) == bad
    assert quant(blocks(dm), q=None, s=None, qt=None, st=None) == bad
    assert quant(blocks(dm), qt=q) == dm.DMUON_ERR_ALIASING
    assert deq(blocks(dm), s=None) == bad


def product(dm, **kw):
    d = dm.dmuon_block_product_t()
    v = dict(m=10, n=200, k=300, lda=300, ldb=300, ldc=200, b_stride=0, experts=0, a_dtype=2, b_dtype=2,
             b_block_rows=128, out_dtype=1, accumulate=0)
    v.update(kw)
    for k, x in v.items():
        setattr(d, k, x)
    return d


def test_block_matmul_refusals(dm):
    M = 1 << 20
    a, sa, b, sb, c = (BASE + i * M for i in range(5))
    bad = dm.DMUON_ERR_INVALID_ARG

    def call(d, a=a, sa=sa, b=b, sb=sb, off=None, c=c):
        return dm._lib.dmuon_block_matmul(d, a, sa, b, sb, off, c, None)

    for kw in (dict(m=-1), dict(n=0), dict(k=0), dict(lda=299), dict(ldb=299), dict(ldc=199), dict(experts=-1),
               dict(b_block_rows=32), dict(accumulate=3), dict(experts=2)):
        assert call(product(dm, **kw)) == bad, kw
    assert call(product(dm), off=BASE + 9 * M) == bad                     # offsets without experts
    assert call(product(dm, experts=2, b_stride=100), off=BASE + 9 * M) == bad
    for kw in (dict(a_dtype=1), dict(b_dtype=0), dict(out_dtype=2)):
        assert call(product(dm, **kw)) == dm.DMUON_ERR_UNSUPPORTED, kw
    for kw in (dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(c=None), dict(c=c + 1),
               dict(sa=sa + 1), dict(sb=sb + 2)):
        assert call(product(dm), **kw) == bad, kw
    assert call(product(dm), c=a) == dm.DMUON_ERR_ALIASING
    assert call(product(dm), c=sb) == dm.DMUON_ERR_ALIASING
    assert call(product(dm, m=0)) == dm.DMUON_OK
    assert call(product(dm, m=1 << 30, n=1 << 22, ldc=1 << 22), sa=1 << 40, b=1 << 50, c=1 << 55) \
        == dm.DMUON_ERR_UNSUPPORTED


def test_binding_refusals(dm):
    import torch
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    x, w, off = torch.zeros(4, 8, dtype=bf), torch.zeros(2, 6, 8, dtype=bf), torch.zeros(3, dtype=torch.int32)
    for args in ((x, w, off.long()), (x, w, off[:2]), (x, w[:, :, :7], off), (x[:, ::2], w[:, :, :4], off),
                 (x.t(), w, off), (x[0], w, off)):
        with pytest.raises(ValueError):
            dm.dmuon_expert_matmul(*args)
    with pytest.raises(ValueError):
        dm.dmuon_expert_matmul(x, w, off)                  # not on a GPU
    with pytest.raises(TypeError):
        dm.dmuon_expert_matmul(x.double(), w.double(), off)
    with pytest.raises(ValueError):
        dm.dmuon_expert_weight_grad(x, x, off, accumulate=True)
    with pytest.raises(ValueError):
        dm.dmuon_quantize_blocks(x, block_rows=64)
    with pytest.raises(KeyError):
        dm.dmuon_quantize_blocks(x, fmt="e3m4")
    q, s = torch.zeros(4, 8, dtype=f8), torch.ones(4, 1)
    for a, sa, b, sb in ((q, s[:3], q, s), (q, s, q[:, :7], s), (q, s, q, s)):
        with pytest.raises(ValueError):
            dm.dmuon_block_matmul(a, sa, b, sb, block_rows=128)
    with pytest.raises(TypeError):
        dm.dmuon_block_matmul(x, s, q, s, block_rows=1)
