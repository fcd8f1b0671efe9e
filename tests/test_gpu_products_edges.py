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
