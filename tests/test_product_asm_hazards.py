"""Wait states around the expert products' matrix instructions.

The 256 x 256 expert kernels issue their matrix instructions as inline asm,
as the 256-tile GEMM does: the same scan of the compiled kernels (a read of an
accumulator needs 19 wait states behind the instruction that wrote it, a write
2 before the one that adds to it) over each of them.  CPU only."""
import os
import shutil
import subprocess

import pytest

from matrix_optimizer_step_owned_amd import _build
from tests.test_gemm_asm_hazards import _hazards

KERNELS = [f"_ZN5dmuon12_GLOBAL__N_122expert_bf16_big_kernelILi{op}E{out}EEvNS_10ExpertArgsE"
           for op, out in ((0, "t"), (1, "t"), (2, "t"), (2, "f"))]


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "experts.s"
    p = subprocess.run([hipcc, *_build.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(_build.CSRC, "experts.hip"),
                        "-o", str(out)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert p.returncode == 0, p.stdout[-4000:]
    return out.read_text().split("\n")


@pytest.mark.parametrize("kernel", KERNELS, ids=["forward", "input", "weight-bf16", "weight-f32"])
def test_no_accumulator_read_inside_mfma_latency(asm, kernel):
    start = next(i for i, l in enumerate(asm) if l.startswith(kernel + ":"))
    end = next(i for i in range(start, len(asm)) if asm[i].startswith(".Lfunc_end"))
    body = [t for t in (l.split(";")[0].strip() for l in asm[start:end])
            if t and (t.endswith(":") or not t.startswith("."))]
    assert sum(t.startswith("v_mfma") for t in body) >= 256, "the kernel's matrix instructions were not found"
    assert not any("scratch_" in t for t in body), "accumulators or fragments in scratch memory"
    found = _hazards(body)
    assert not found, "\n".join(found[:20])
