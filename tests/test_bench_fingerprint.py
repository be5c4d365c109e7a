"""The fingerprint that pins counters to a workload's kernel covers every file
that the kernel's code and launch rules stand in."""
import os
import shutil
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402

RING = [w for w, k in bench.KERNEL_NAMES.items() if k.startswith("k_gemm_dma")]


@pytest.mark.parametrize("workload", RING)
@pytest.mark.parametrize("changed", ["gemm_ring.hpp", "k_gemm_dma.hip", "dev_common.hpp"])
def test_ring_workloads(monkeypatch, tmp_path, workload, changed):
    csrc = os.path.join("conv_qgemm_amd", "csrc")
    shutil.copytree(os.path.join(ROOT, csrc), tmp_path / csrc)
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    before = bench.src_sha(bench.KERNEL_SOURCES[workload])
    with open(tmp_path / csrc / changed, "a") as f:
        f.write("// only a comment\n")
    assert bench.src_sha(bench.KERNEL_SOURCES[workload]) == before
    with open(tmp_path / csrc / changed, "a") as f:
        f.write("int another_line;\n")
    assert bench.src_sha(bench.KERNEL_SOURCES[workload]) != before
