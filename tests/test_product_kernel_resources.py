"""What the compiler made of the expert and block kernels (CPU only): no kernel
keeps registers in scratch memory, and the few-rows kernels exist only in the
forms that some call launches."""
import os
import re
import shutil
import subprocess

import pytest

from matrix_optimizer_step_owned_amd import _build

LLVM = "/opt/rocm/llvm/bin"


def _kernels(name, tmp):
    """{kernel: metadata} of one compiled source, taken from build()'s object
    or, where there is none, compiled here."""
    if not os.path.exists(os.path.join(LLVM, "llvm-readelf")):
        pytest.skip("no LLVM tools")
    obj = os.path.join(_build.BUILD, name + ".o")
    if not os.path.exists(obj):
        hipcc = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
        obj = str(tmp / (name + ".o"))
        subprocess.run([hipcc, *_build.HIPCC_FLAGS, "-c", os.path.join(_build.CSRC, name + ".hip"), "-o", obj],
                       check=True, capture_output=True)
    fat, code = str(tmp / (name + ".fat")), str(tmp / (name + ".co"))
    subprocess.run([f"{LLVM}/llvm-objcopy", f"--dump-section=.hip_fatbin={fat}", obj, os.devnull], check=True)
    subprocess.run([f"{LLVM}/clang-offload-bundler", "--unbundle", "--type=o",
                    "--targets=hipv4-amdgcn-amd-amdhsa--gfx950", f"--input={fat}", f"--output={code}"], check=True)
    notes = subprocess.run([f"{LLVM}/llvm-readelf", "--notes", code], check=True, capture_output=True, text=True).stdout
    out = {}
    for part in re.split(r"\n\s+\.name:\s+(?=_ZN5dmuon)", notes)[1:]:
        get = lambda key: int(re.search(rf"\.{key}:\s+(\d+)", part).group(1))
        out[part.split()[0]] = {k: get(k) for k in ("private_segment_fixed_size", "vgpr_spill_count")}
    assert out
    return out


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("objects")
    return {name: _kernels(name, tmp) for name in ("experts", "blocks")}


@pytest.mark.parametrize("source", ["experts", "blocks"])
def test_no_scratch_memory(kernels, source):
    bad = {k: v for k, v in kernels[source].items() if any(v.values())}
    assert not bad, bad


def test_few_rows_forms(kernels):
    """(row blocks, column blocks, waves[, result]): sixteen waves only for one
    block of rows by one of columns and bf16 results."""
    forms = lambda source, tail: sorted(m.groups() for m in (
        re.search(r"skinny_kernelILi(\d)ELi(\d)ELi(\d+)E" + tail, k) for k in kernels[source]) if m)
    assert forms("experts", "E") == [("1", "1", "16"), ("1", "1", "8"), ("1", "2", "8"), ("2", "2", "8")]
    assert forms("blocks", "([ft])E") == [("1", "1", "16", "t"), ("1", "1", "8", "f"), ("1", "1", "8", "t"),
                                         ("1", "2", "8", "f"), ("1", "2", "8", "t"), ("2", "2", "8", "f"),
                                         ("2", "2", "8", "t")]
