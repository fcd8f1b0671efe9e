"""The Python binding of the expert products and the 8-bit block operators (CPU)."""
import os
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_without_the_raw_stream_getter():
    """A build of PyTorch that lacks the private stream getter still imports
    the package and plans on the host."""
    code = ("import torch\n"
            "if hasattr(torch._C, '_cuda_getCurrentRawStream'):\n"
            "    del torch._C._cuda_getCurrentRawStream\n"
            "import matrix_optimizer_step_owned_amd as dm\n"
            "assert dm.dmuon_plan_describe([(64, 128)])\n"
            "assert dm.dmuon_assign_owners([(64, 128), (32, 32)], 2)\n")
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                       text=True)
    assert p.returncode == 0, p.stdout[-2000:]


def _calls(dm):
    """Every entry point as a call of one tensor that requires a gradient and
    others that do not, by the operand that requires it."""
    bf, f8 = torch.bfloat16, torch.float8_e4m3fn
    x, w, dy = torch.zeros(4, 8, dtype=bf), torch.zeros(2, 6, 8, dtype=bf), torch.zeros(4, 6, dtype=bf)
    off, q, s = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8, dtype=f8), torch.ones(4, 1)
    return {
        "matmul x": lambda r: dm.dmuon_expert_matmul(r(x), w, off),
        "matmul w": lambda r: dm.dmuon_expert_matmul(x, r(w), off),
        "matmul out": lambda r: dm.dmuon_expert_matmul(x, w, off, out=r(dy)),
        "input grad dy": lambda r: dm.dmuon_expert_input_grad(r(dy), w, off),
        "input grad w": lambda r: dm.dmuon_expert_input_grad(dy, r(w), off),
        "weight grad dy": lambda r: dm.dmuon_expert_weight_grad(r(dy), x, off),
        "weight grad x": lambda r: dm.dmuon_expert_weight_grad(dy, r(x), off),
        "weight grad out": lambda r: dm.dmuon_expert_weight_grad(dy, x, off, out=r(w), accumulate=True),
        "quantise": lambda r: dm.dmuon_quantize_blocks(r(x)),
        "dequantise": lambda r: dm.dmuon_dequantize_blocks(q, r(s)),
        "block matmul scale": lambda r: dm.dmuon_block_matmul(q, r(s), q, s, block_rows=1),
        "block matmul out": lambda r: dm.dmuon_block_matmul(q, s, q, s, block_rows=1, out=r(torch.zeros(4, 4, dtype=bf))),
    }


@pytest.mark.parametrize("call", ["matmul x", "matmul w", "matmul out", "input grad dy", "input grad w",
                                  "weight grad dy", "weight grad x", "weight grad out", "quantise", "dequantise",
                                  "block matmul scale", "block matmul out"])
def test_no_gradient_is_lost_in_silence(call):
    """No call records a graph, so a tensor that requires a gradient is refused
    where one would be recorded; elsewhere the call goes on (to the check that
    finds the CPU's tensors)."""
    import matrix_optimizer_step_owned_amd as dm
    f = _calls(dm)[call]
    wants = lambda t: t.clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        f(wants)
    with torch.no_grad(), pytest.raises(ValueError, match="GPU"):
        f(wants)
    with pytest.raises(ValueError, match="GPU"):
        f(lambda t: t)


def test_one_row_of_any_stride():
    """The last token of a long prompt is one row with the prompt's stride,
    which no access uses: rows of 2^22 elements and more apart are taken."""
    import matrix_optimizer_step_owned_amd as dm
    far = torch.empty_strided((1, 64), (1 << 24, 1), dtype=torch.bfloat16)
    assert dm._rows2(far, "x") == (1, 64, 64)
    assert dm._rows2(far[:0], "x") == (0, 64, 64)
    assert dm._rows2(torch.empty(5, 80)[:, :64], "x") == (5, 64, 80)


def test_transpose_alone_refusals():
    import matrix_optimizer_step_owned_amd as dm
    x, q, s = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.float8_e4m3fn), torch.zeros(4, 1)
    for kw in (dict(), dict(transposed=True, q=q), dict(transposed=True, scale=s)):
        with pytest.raises(ValueError, match="plain"):
            dm.dmuon_quantize_blocks(x, plain=False, **kw)
