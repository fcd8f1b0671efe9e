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
