"""Attention over more widened tiles than the workspace has room for at a time:
the batch runs in slices of its sequences, with the results of smaller batches."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def test_slices_of_a_batch():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from conv_qgemm_amd import qgemm as qg
    S, H, Hq, D, bs, n, L = 72, 16, 64, 256, 64, 260, 900
    size = qg.lib.qattn_kv8_workspace_size
    assert 2 * size(S // 2 * n, S // 2, n, L, Hq, H, D) > 1 << 30 >= size(S * n, S, n, L, Hq, H, D)
    g = torch.Generator(device="cuda").manual_seed(5)
    need = -(-L // bs)

    def codes():
        return torch.randint(-127, 128, (S * need, H, bs, D), dtype=torch.int8, device="cuda", generator=g)

    def scales():
        return torch.rand(S * need, H, device="cuda", generator=g) * 0.02 + 0.01

    cache = qg.KVCache(codes(), codes(), scales(), scales())
    table = torch.randperm(S * need, device="cuda", generator=g).int().view(S, need)
    lens = torch.tensor([L - 7 * (i % 80) for i in range(S)], dtype=torch.int32, device="cuda")
    q = torch.randn(S * n, Hq, D, device="cuda", generator=g).to(torch.bfloat16)

    def call(b0, b1):
        cu = torch.arange(0, (b1 - b0) * n + 1, n, dtype=torch.int32, device="cuda")
        return qg.qattn_kv8(q[b0 * n:b1 * n], cache, table[b0:b1], cu, lens[b0:b1].contiguous(), n, L,
                            return_lse=True)

    print(f"slices: {S} sequences of {n} new tokens", flush=True)
    out, lse = call(0, S)
    for b0 in (0, S // 2):
        some, some_lse = call(b0, b0 + S // 2)
        at = slice(b0 * n, (b0 + S // 2) * n)
        assert torch.equal(out[at], some) and torch.equal(lse[at], some_lse)
