"""Sequences that share the blocks of a common prefix, and go on in blocks of
their own: what is read and attended over is as if each had its own copy."""
import numpy as np
import pytest

from oracle import kv8

from test_gpu_kv_cache import as_cache, dev, make_cache, new_values

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("new", [1, 3, 40])
def test_shared_prefix(new):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from conv_qgemm_amd import qgemm as qg
    rng = np.random.default_rng(2)
    S, H, Hq, D, bs = 3, 2, 8, 64, 16
    shared, own = [5, 2, 9], 4                       # three whole blocks, then their own
    pool = 10 + S * own
    start = make_cache(rng, pool, H, bs, D)
    table = np.array([shared + [10 + own * i + j for j in range(own)] for i in range(S)], np.int32)
    kv = [48 + new, 48 + 5 + new, 48 + 15 + new]     # some own blocks begun earlier
    cu = np.arange(S + 1, dtype=np.int32) * new
    x = new_values(rng, S * new, Hq + 2 * H, D, "bf16")
    xf = x.float().numpy()
    c = as_cache(qg, start)
    tab, cud, lens = dev(table), dev(cu), dev(np.array(kv, np.int32))
    xd = x.cuda()
    print(f"shared prefix, {new} new tokens", flush=True)
    q = qg.qkv_append_rope(xd[:, :Hq], xd[:, Hq:Hq + H], xd[:, Hq + H:], c, tab, cud, lens, new)
    total = np.concatenate([[0], np.cumsum(kv)]).astype(np.int32)
    k, v = qg.qkv_read(c, tab, torch.zeros_like(lens), dev(total), int(total[-1]), dtype=torch.float32)
    out, lse = qg.qattn_kv8(q, c, tab, cud, lens, new, max(kv), return_lse=True)
    kv8.append(xf[:, Hq:Hq + H], xf[:, Hq + H:], start, table, cu, kv)
    for got, want in zip(c, start):
        assert np.array_equal(got.cpu().numpy(), want)
    wk, wv = kv8.read(start, table, [0] * S, kv)
    assert np.array_equal(k.cpu().numpy(), wk) and np.array_equal(v.cpu().numpy(), wv)
    # copies of the prefix for each sequence: the same bits
    apart = np.arange(S * (3 + own), dtype=np.int32).reshape(S, -1)
    copies = [dev(a[table].reshape(-1, *a.shape[1:])) for a in start]
    out2, lse2 = qg.qattn_kv8(q, qg.KVCache(*copies), dev(apart), cud, lens, new, max(kv),
                              return_lse=True)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
