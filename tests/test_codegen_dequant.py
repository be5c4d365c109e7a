"""The generated-code guards of the large-GEMM kernel on its float-output forms
(k_gemm_dma_dequant.hip): accumulators out of scratch, the ring's loads in
flight, the loop's shape; and 16-bit results rounded in two steps."""
import os
import re
import subprocess

import pytest

import test_codegen


@pytest.fixture(scope="module")
def asm(tmp_path_factory):
    from conv_qgemm_amd import build
    src = "k_gemm_dma_dequant.hip"
    out = tmp_path_factory.mktemp("asm") / (src + ".s")
    cmd = [build.HIPCC, *build.flags_for(src), "--cuda-device-only", "-S",
           os.path.join(build.CSRC, src), "-o", str(out)]
    subprocess.run(cmd, check=True, capture_output=True)
    return out.read_text()


# three output types, each stage by stage and in pairs of stages
@pytest.mark.parametrize("guard", ["test_no_scratch", "test_main_loop_shape", "test_accumulators_not_spilled"])
def test_guards(monkeypatch, asm, guard):
    monkeypatch.setattr(test_codegen, "N_INSTANTIATIONS", 6)
    getattr(test_codegen, guard)(asm)


def test_private_memory(asm):
    """Three values of the prologue, read again once per tile; nothing else."""
    sizes = re.findall(r"\.private_segment_fixed_size:\s+(\d+)", asm)
    assert len(sizes) == 6 and all(int(s) <= 16 for s in sizes), sizes
    assert len(re.findall("scratch_load", asm)) <= 3 * 6


def test_no_mixed_precision_rounding(asm):
    assert not re.search(r"v_(fma|mad)_mix", asm)
