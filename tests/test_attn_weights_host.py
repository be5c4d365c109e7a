"""The attention kernels' scale factors on the host: they are compiled on the
promise that no operation makes a NaN, so blocks of zeros (scale 0) must not
make one on the way to a result either."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_no_invalid_operation_for_any_scale(tmp_path):
    exe = tmp_path / "check"
    subprocess.run(["g++", "-O1", "-frounding-math", "-ftrapping-math", "-std=c++17",
                    "-I" + os.path.join(ROOT, "conv_qgemm_amd", "csrc"),
                    os.path.join(ROOT, "tests", "c", "attn_weights_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
