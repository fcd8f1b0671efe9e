"""Expert products and 8-bit blocks on the GPU where a call leaves the
ordinary path: streams, single rows of any stride, padded rows, non-finite
neighbours, sums that cancel."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def test_stream_handle_without_the_raw_getter(lib, monkeypatch):
    """The public way to the current stream's handle gives the private one's,
    and calls go there."""
    side = torch.cuda.Stream()
    x, w = torch.ones(3, 16, dtype=BF, device=DEV), torch.ones(1, 8, 16, dtype=BF, device=DEV)
    offs = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            assert lib._current_stream(0) == lib._raw_stream(0) == stream.cuda_stream
    monkeypatch.setattr(lib, "_raw_stream", lib._current_stream)
    with torch.cuda.stream(side):
        y = lib.dmuon_expert_matmul(x, w, offs)
    side.synchronize()
    assert bool((y == 16).all())


class _Experts(torch.autograd.Function):
    """The three products joined as their documentation says."""

    @staticmethod
    def forward(ctx, lib, x, w, offs):
        ctx.lib = lib
        ctx.save_for_backward(x, w, offs)
        return lib.dmuon_expert_matmul(x, w, offs)

    @staticmethod
    def backward(ctx, dy):
        x, w, offs = ctx.saved_tensors
        dy = dy.contiguous()
        return None, ctx.lib.dmuon_expert_input_grad(dy, w, offs), ctx.lib.dmuon_expert_weight_grad(dy, x, offs), None


def test_products_inside_an_autograd_function(lib):
    """The gradients that autograd hands on are the gradient products'; the
    bare call refuses the same tensors."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(30, 24, generator=g, device=DEV).requires_grad_()
    w = torch.randn(2, 16, 24, generator=g, device=DEV).requires_grad_()
    offs = torch.tensor([0, 11, 30], dtype=torch.int32, device=DEV)
    y = _Experts.apply(lib, x, w, offs)
    dy = torch.randn(30, 16, generator=g, device=DEV)
    y.backward(dy)
    with torch.no_grad():
        assert torch.equal(x.grad, lib.dmuon_expert_input_grad(dy, w, offs))
        assert torch.equal(w.grad, lib.dmuon_expert_weight_grad(dy, x, offs))
    with pytest.raises(ValueError, match="gradient"):
        lib.dmuon_expert_matmul(x, w, offs)


def test_one_row_of_a_long_prompt(lib):
    """hidden[:, -1] of one sequence: a row with a stride above 2^22."""
    g = torch.Generator(device=DEV).manual_seed(2)
    k, n = 1024, 64
    x = torch.randn(1, 4200, k, generator=g, device=DEV).to(BF)[:, -1]
    assert x.stride(0) > 1 << 22 and x.data_ptr() % 16 == 0
    w = torch.randn(1, n, k, generator=g, device=DEV).to(BF)
    dy = torch.randn(1, 70000, n, generator=g, device=DEV).to(BF)[:, -1]
    offs = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    flat, dflat = x.clone(), dy.clone()
    assert torch.equal(lib.dmuon_expert_matmul(x, w, offs), lib.dmuon_expert_matmul(flat, w, offs))
    assert torch.equal(lib.dmuon_expert_input_grad(dy, w, offs), lib.dmuon_expert_input_grad(dflat, w, offs))
    assert torch.equal(lib.dmuon_expert_weight_grad(dy, x, offs), lib.dmuon_expert_weight_grad(dflat, flat, offs))
    q, s, qt, st = lib.dmuon_quantize_blocks(x, transposed=True)
    want = lib.dmuon_quantize_blocks(flat, transposed=True)
    assert all(torch.equal(a.float(), b.float()) for a, b in zip((q, s, qt, st), want))
    out = torch.zeros(1, 70000, n, dtype=BF, device=DEV)
    wq, ws, _, _ = lib.dmuon_quantize_blocks(w[0], block_rows=128)
    y = lib.dmuon_block_matmul(q, s, wq, ws, out=out[:, -1])
    assert torch.equal(y, lib.dmuon_block_matmul(q, s, wq, ws))
    assert not bool(out[:, :-1].any())


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_transpose_alone(lib, block_rows, dtype):
    """The quantised transpose without the plain copy is the pair's."""
    g = torch.Generator(device=DEV).manual_seed(3)
    for shape in ((1, 1), (130, 257), (3, 64, 384)):
        x = torch.randn(shape, generator=g, device=DEV).to(dtype)
        _, _, qt, st = lib.dmuon_quantize_blocks(x, block_rows=block_rows, transposed=True)
        none, none_s, got, scale = lib.dmuon_quantize_blocks(x, block_rows=block_rows, transposed=True, plain=False)
        assert none is None and none_s is None
        assert torch.equal(got.float(), qt.float()) and torch.equal(scale, st)
        got.view(torch.uint8).zero_()
        lib.dmuon_quantize_blocks(x, block_rows=block_rows, plain=False, qt=got, scale_t=scale)
        assert torch.equal(got.float(), qt.float())


def test_more_than_2_31_elements(lib):
    """264192 rows of 8192: the last rows of every result against the same rows
    alone.  Tolerances: sums of `length` products in fp32, (length + 2) 2^-24 of
    their magnitudes and half a bf16 step; the 8-bit product against the
    fp32-result one, whose operands are the same: at most 8 * 2^-13 of the largest
    product of every eight, bounded by the rows' largest values."""
    t, k, n, last = 264192, 8192, 16, 256
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.empty(t, k, dtype=BF, device=DEV).normal_(generator=g)
    assert x.numel() > 1 << 31
    w = (torch.randn(1, n, k, generator=g, device=DEV) * 0.05).to(BF)
    offs = torch.tensor([0, t], dtype=torch.int32, device=DEV)
    tail, W = x[-last:].double(), w[0].double()
    mag = tail.abs() @ W.abs().t().contiguous()
    y = lib.dmuon_expert_matmul(x, w, offs)
    ref = tail @ W.t().contiguous()
    assert bool(((y[-last:].double() - ref).abs() <= (k + 2) * 2.0 ** -24 * mag + 2.0 ** -8 * (1 + 2.0 ** -9) * ref.abs()).all())
    dx = lib.dmuon_expert_input_grad(x, w.view(1, k, n), offs)       # x as the gradient of 8192 outputs
    V = w.view(k, n).double()
    ref = tail @ V
    tol = (k + 2) * 2.0 ** -24 * (tail.abs() @ V.abs()) + 2.0 ** -8 * (1 + 2.0 ** -9) * ref.abs()
    assert bool(((dx[-last:].double() - ref).abs() <= tol).all())
    only = torch.tensor([t - last, t], dtype=torch.int32, device=DEV)
    dw = lib.dmuon_expert_weight_grad(y, x, only, out_dtype=F32)[0]
    D = y[-last:].double().t().contiguous()
    assert bool(((dw.double() - D @ tail).abs() <= (last + 2) * 2.0 ** -24 * (D.abs() @ tail.abs())).all())
    q, s, qt, st = lib.dmuon_quantize_blocks(x, transposed=True)
    for got, want in zip((q[-last:], s[-last:], qt[:, -last:], st[:, -last // 128:]),
                         lib.dmuon_quantize_blocks(x[-last:], transposed=True)):
        assert torch.equal(got.float(), want.float())
    del qt, st
    back = lib.dmuon_dequantize_blocks(q, s)
    assert torch.equal(back[-last:], lib.dmuon_dequantize_blocks(q[-last:], s[-last:]))
    del back, x
    wq, ws, _, _ = lib.dmuon_quantize_blocks(w[0], block_rows=128)
    got = lib.dmuon_block_matmul(q, s, wq, ws)[-last:].double()
    full = lib.dmuon_block_matmul(q, s, wq, ws, out_dtype=F32)[-last:].double()
    alone = lib.dmuon_block_matmul(q[-last:], s[-last:], wq, ws, out_dtype=F32).double()
    A, B = lib.dmuon_dequantize_blocks(q[-last:], s[-last:], dtype=F32), lib.dmuon_dequantize_blocks(wq, ws, block_rows=128, dtype=F32)
    mag = A.double().abs() @ B.double().abs().t().contiguous()
    assert bool(((full - alone).abs() <= 2 * (k + 3 * 64 + 3) * 2.0 ** -24 * mag).all())
    tol = torch.zeros_like(mag)
    for c in range(0, k, 8):
        tol += 8 * 2.0 ** -13 * torch.outer(A[:, c:c + 8].abs().amax(1).double(), B[:, c:c + 8].abs().amax(1).double())
    tol += (2 * k // 8 + 2 * (k + 3 * 64 + 3)) * 2.0 ** -24 * mag
    assert bool(((got - full).abs() <= tol + 2.0 ** -8 * (full.abs() + tol)).all())


@pytest.mark.parametrize("tokens,n,k", [(720, 8200, 208), (20, 264, 528), (40, 1800, 144)],
                         ids=["large-tiles", "few-rows", "few-rows-wide"])
def test_replays(lib, tokens, n, k):
    """The large-tile and few-rows kernels captured into a graph and replayed with
    other offsets and values, eager calls between the replays: bit for bit."""
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn(tokens, k, generator=g, device=DEV).to(BF)
    dy = torch.randn(tokens, n, generator=g, device=DEV).to(BF)
    w = torch.randn(5, n, k, generator=g, device=DEV).to(BF)
    offs = torch.zeros(6, dtype=torch.int32, device=DEV)
    y, y8 = torch.zeros(tokens, n, dtype=BF, device=DEV), torch.zeros(tokens, n, dtype=BF, device=DEV)
    y32, dw = torch.zeros(tokens, n, device=DEV), torch.zeros(5, n, k, device=DEV)
    xq, xs, _, _ = lib.dmuon_quantize_blocks(x)
    wq, ws, _, _ = lib.dmuon_quantize_blocks(w, block_rows=128)
    outs = (y, y8, y32, dw, xq, xs)

    def go():
        lib.dmuon_expert_matmul(x, w, offs, out=y)
        lib.dmuon_expert_weight_grad(dy, x, offs, out=dw, accumulate=True)
        lib.dmuon_quantize_blocks(x, q=xq, scale=xs)
        lib.dmuon_block_matmul(xq, xs, wq, ws, offsets=offs, out=y8)
        lib.dmuon_block_matmul(xq, xs, wq, ws, offsets=offs, out=y32)

    def start():
        for t in (y, y8, y32, dw):
            t.zero_()

    go()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for new in ([0, 1, 1, 5, 9, tokens], [2] * 6, [0, 0, tokens, tokens, tokens, tokens], [1, 4, 7, 9, 12, tokens - 1]):
        offs.copy_(torch.tensor(new, dtype=torch.int32))
        x.mul_(-0.75)
        start()
        go()
        torch.cuda.synchronize()
        want = [t.float().clone() for t in outs]
        start()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t.float(), v) for t, v in zip(outs, want)), new
