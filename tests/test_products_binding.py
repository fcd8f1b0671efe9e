"""The Python binding of the expert products and the 8-bit block operators (CPU)."""
import os
import subprocess
import sys

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
