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
