"""New queries whose sequences hold no token at all: 0 and -infinity, whatever
kernel their number picks."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("n", [[1], [1, 1, 2], [40], [300], [1100, 3], [2000]])
def test_empty_cache(n, causal):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from conv_qgemm_amd import qgemm as qg
    cache = qg.kv_cache(2, 1, 16, 64)
    table = torch.full((len(n), 1), -1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + n, device="cuda").cumsum(0).int()
    lens = torch.zeros(len(n), dtype=torch.int32, device="cuda")
    q = torch.randn(sum(n), 4, 64, device="cuda").to(torch.bfloat16)
    print(f"empty cache, {n} new tokens", flush=True)
    for max_kv in (0, 5):
        out, lse = qg.qattn_kv8(q, cache, table, cu, lens, max(n), max_kv, causal=causal, return_lse=True)
        assert not out.any() and torch.isneginf(lse).all()
