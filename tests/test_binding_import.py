"""The binding without the module of the decoding step's calls (_qcall.so, built
for one interpreter and one torch): the calls that need only ctypes are there,
the others say what is missing.  In a process of its own, on the host."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import sys
sys.modules["conv_qgemm_amd._qcall"] = None  # an import of it fails
import torch
from conv_qgemm_amd import qgemm as qg
assert qg.version() > 0
assert qg.lib.qgemm_s8s8_requant(None, 0, None, 0, None, None, None, None, 0, 0, 0, 0, None) == qg.QG_ERR_NULLPTR
a = torch.zeros(1, 16, dtype=torch.int8)
i = torch.zeros(1, dtype=torch.int32)
try:
    qg.qgemm_s8s8_requant(a, a, i, i, i)
    raise SystemExit("a host tensor was taken")
except ValueError as e:
    assert "GPU tensor" in str(e)
t, x = torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1, 64, dtype=torch.bfloat16)
c = qg.kv_cache(1, 1, 16, 64, device="cpu")
for call in (lambda: qg.qgemm_s8s8_dequant(a, a), lambda: qg.qkv_append_rope(None, x, x, c, t, i, i, 1),
             lambda: qg.qkv_read(c, t, i, i, 1), lambda: qg.qattn_kv8(x, c, t, i, i, 1, 1)):
    try:
        call()
        raise SystemExit("a call without its module")
    except ImportError as e:
        assert "_qcall.so" in str(e) and "build" in str(e)
print("ok")
"""


def test_older_calls_need_only_ctypes():
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stderr[-2000:]


def test_library_is_linked_before_the_module(monkeypatch, tmp_path):
    """A torch without its headers costs the module, not the library."""
    from conv_qgemm_amd import build
    linked = []
    monkeypatch.setattr(build, "_compile", lambda src: str(tmp_path / src))
    monkeypatch.setattr(build, "_link", lambda objs, lib, *a, **k: linked.append(lib))

    def no_headers(verbose):
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(build, "_build_call", no_headers)
    try:
        build.build()
        raise AssertionError("a failed module went unnoticed")
    except RuntimeError as e:
        assert "g++ failed" in str(e)
    assert linked[0] == build.LIB and len(linked) == 3
