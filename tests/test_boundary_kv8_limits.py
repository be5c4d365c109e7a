"""The limits that the header states for the int8 cache's calls: sizes at them
pass the checks (and stop at the missing device), sizes past them do not."""
import pytest

from test_boundary_kv8 import ap, at, qg, rd  # noqa: F401


@pytest.fixture(scope="module")
def ok(qg):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("needs a machine without a GPU")
    return qg.QG_ERR_NO_DEVICE


def both(qg, ok, call, good, bad):  # noqa: F811
    assert call(qg, **good) == ok, good
    assert call(qg, **{**good, **bad}) == qg.QG_ERR_INVALID, bad


def test_append(qg, ok):  # noqa: F811
    # (tokens / 16 + 2 seqs) * heads * 2 + tokens < 2^24
    wide = dict(H=1, Hq=1, ldk=64, ldv=64, ldq=64, ldqo=64, seqs=1, max_q=5)
    top = max(t for t in range(14912000, 14913200) if (t // 16 + 2) * 2 + t < 1 << 24)
    both(qg, ok, ap, dict(wide, tokens=top), dict(tokens=top + 1))
    seqs = dict(H=8, Hq=8, ldk=512, ldv=512, ldq=512, ldqo=512, tokens=0x10, max_q=5)
    both(qg, ok, ap, dict(seqs, seqs=(1 << 19) - 2), dict(seqs=1 << 19))


def test_read(qg, ok):  # noqa: F811
    both(qg, ok, rd, dict(tokens=(1 << 24) - 1), dict(tokens=1 << 24))


def test_attention(qg, ok):  # noqa: F811
    # rows * heads / 16 decide: 2^24 less one sequence's item
    one = dict(H=1, Hq=1, ldq=64, ldo=64, seqs=1, max_q=1 << 28, max_kv=16)
    both(qg, ok, at, dict(one, tokens=(1 << 28) - 32), dict(tokens=(1 << 28) - 16))
    # sequences: (rows / 128 + seqs) * heads < 2^23
    many = dict(H=8, Hq=8, ldq=512, ldo=512, tokens=100, max_q=1, max_kv=16)
    both(qg, ok, at, dict(many, seqs=(1 << 20) - 1), dict(seqs=1 << 20))


def test_common(qg, ok):  # noqa: F811
    for call in (ap, rd, at):
        both(qg, ok, call, dict(bs=128, cols=1 << 23, ldt=1 << 23), dict(cols=(1 << 23) + 1, ldt=(1 << 23) + 1))
