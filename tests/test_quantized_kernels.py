"""What the compiler made of the kernels on 8-bit states, 8-bit integers and of the expert layer
(CPU only): no registers in scratch memory; in the 256 x 256 product of 8-bit integers, whose matrix
instructions are inline asm, no accumulator is read inside their latency."""
import os
import shutil
import subprocess

import pytest

from matrix_optimizer_step_owned_amd import _build
from tests.test_gemm_asm_hazards import _hazards
from tests.test_product_kernel_resources import _kernels


@pytest.mark.parametrize("source", ["adamw8", "int8", "layer"])
def test_no_scratch_memory(source, tmp_path):
    bad = {k: v for k, v in _kernels(source, tmp_path).items() if any(v.values())}
    assert not bad, bad


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("asm") / "int8.s"
    p = subprocess.run([hipcc, *_build.HIPCC_FLAGS, "--cuda-device-only", "-S", os.path.join(_build.CSRC, "int8.hip"),
                        "-o", str(out)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert p.returncode == 0, p.stdout[-4000:]
    return out.read_text().split("\n")


@pytest.mark.parametrize("out", ["t", "f"], ids=["bf16", "f32"])
def test_no_accumulator_read_inside_mfma_latency(asm, out):
    kernel = f"_ZN5dmuon12_GLOBAL__N_122int8_matmul_big_kernelI{out}EEvNS_8Int8ArgsE"
    start = next(i for i, l in enumerate(asm) if l.startswith(kernel + ":"))
    end = next(i for i in range(start, len(asm)) if asm[i].startswith(".Lfunc_end"))
    body = [t for t in (l.split(";")[0].strip() for l in asm[start:end])
            if t and (t.endswith(":") or not t.startswith("."))]
    assert sum(t.startswith("v_mfma_i32_16x16x64_i8 a[") for t in body) >= 256
    assert not any("scratch_" in t for t in body)
    found = _hazards(body)
    assert not found, "\n".join(found[:20])
