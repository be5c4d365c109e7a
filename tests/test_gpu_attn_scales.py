"""Attention over the int8 cache (qattn_kv8) where the cache's value scales lie
far apart, against binary64: a row's error is bounded by the row's own terms,
whatever the scales of tokens that it does not see or hardly weighs.

Tolerances, from the arithmetic and fixed before the first run.  With u the unit
roundoff of the type (2^-8 bfloat16, 2^-11 binary16), p the softmax, s the value
scales, A = sum_j p_j |v_j| and L the length:
  |out - out64| <= 1.01 (u |out64| + 2^-11 A) + 4 e A + tail
  |lse - lse64| <= e + 2^-20 (1 + |lse64|)
2^-11 A: the coarsest weights are single binary16 numbers.  e is the error of a
score: D products summed in binary32 (2 D 2^-24 scale max_j sum_d |q_d k_jd|),
scaling, exponential and running sums (2^-18), and the scales' logarithms, which
pass through four additions of numbers up to their span (4 * 2^-24 * span).
tail = L 2^-31 * 127 max_j p_j s_j: a weight times its scale is kept to 2^-25 of
binary16's unit, where the largest of the row is at least 2^6."""
import numpy as np
import pytest

from test_gpu_kv_cache import as_cache, dev, make_cache, make_table

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def qg():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from conv_qgemm_amd import qgemm
    return qgemm


def plain(q, cache, table, cu, kv, scale, causal):
    """out, lse, A, max_j p_j s_j and the scores' size, in binary64."""
    T, Hq, D = q.shape
    H, bs = cache[0].shape[1:3]
    G = Hq // H
    out, A = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, top, dot = np.full((T, Hq), -np.inf), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b, L in enumerate(kv):
        t0, n = cu[b], cu[b + 1] - cu[b]
        if n == 0 or L == 0:
            continue
        blk, at = table[b, np.arange(L) // bs], np.arange(L) % bs
        sees = np.minimum(L, L - n + np.arange(n) + 1) if causal else np.full(n, L)
        hidden = np.arange(L)[None] >= sees[:, None]
        for h in range(Hq):
            k = cache[0][blk, h // G, at].astype(float) * cache[2][blk, h // G][:, None].astype(float)
            s = cache[3][blk, h // G].astype(float)
            v = cache[1][blk, h // G, at].astype(float) * s[:, None]
            x = q[t0:t0 + n, h] @ k.T * scale
            x[hidden] = -np.inf
            m = x.max(1)
            some = np.isfinite(m)
            w = np.exp(x - np.where(some, m, 0)[:, None])
            z = np.where(some, w.sum(1), 1)
            p = w / z[:, None]
            out[t0:t0 + n, h], A[t0:t0 + n, h] = p @ v, p @ np.abs(v)
            lse[t0:t0 + n, h] = np.where(some, m + np.log(z), -np.inf)
            top[t0:t0 + n, h] = (p * s).max(1)
            dot[t0:t0 + n, h] = (np.abs(q[t0:t0 + n, h]) @ np.abs(k).T * scale).max(1)
    return out, lse, A, top, dot


def check(qg, q_lens, kv, Hq, H, D, bs, dtype, scales, causal=True, quiet=None, max_kv=None):
    """scales(blocks of a sequence) gives their value scales; keys of the tokens
    that quiet(block, blocks) names score about 40 below the others."""
    rng = np.random.default_rng(7)
    pool = sum(-(-x // bs) for x in kv) + 2
    cache = make_cache(rng, pool, H, bs, D)
    for i in (0, 1):
        cache[i] = np.clip(np.rint(rng.normal(size=cache[i].shape) * 36), -127, 127).astype(np.int8)
    table = make_table(rng, kv, bs, pool)
    T = sum(q_lens)
    cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = rng.normal(size=(T, Hq, D))
    if quiet:  # the first quarter of a head turns against quiet keys
        q[..., :D // 4] = 1.0
    q = torch.from_numpy(q).to(DTYPES[dtype])
    span = 16.0
    for b in range(len(kv)):
        n = -(-kv[b] // bs)
        f = np.asarray(scales(n), np.float32)
        cache[3][table[b, :n]] = f[:, None]
        for x in (0, 1, 2, 3):  # blocks of zeros
            cache[x][table[b, :n][f == 0]] = 0
        if (f > 0).any():
            e2 = np.log2(f[f > 0].astype(float))
            span = max(span, 16 + e2.max() - e2.min())
        for i in range(n):
            if quiet and quiet(i, n):
                # 127 * D / 4 * ks / sqrt(D) = 40
                cache[0][table[b, i], :, :, :D // 4] = -127
                cache[2][table[b, i]] = 40 * 4 / 127 * D ** -0.5
    print(f"scales q={q_lens[:6]} kv={kv[:6]} Hq={Hq} H={H} D={D} bs={bs} {dtype} causal={causal}",
          flush=True)
    out, lse = qg.qattn_kv8(q.cuda(), as_cache(qg, cache), dev(table), dev(cu), dev(np.array(kv, np.int32)),
                            max(q_lens), max(kv) if max_kv is None else max_kv, causal=causal,
                            return_lse=True)
    want, wlse, A, top, dot = plain(q.double().numpy(), cache, table, cu, kv, D ** -0.5, causal)
    e = 2 * D * 2.0 ** -24 * dot + 2.0 ** -18 + 4 * 2.0 ** -24 * span
    tol = 1.01 * (U[dtype] * np.abs(want) + 2.0 ** -11 * A) + 4 * e[..., None] * A + \
        (max(kv) * 2.0 ** -31 * 127 * top)[..., None]
    if dtype == "f16":  # results below binary16's normal range are multiples of 2^-24
        tol = tol + 2.0 ** -25
    got, glse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4], bad.mean())
    seen = np.isfinite(wlse)
    assert np.array_equal(np.isneginf(glse), ~seen) and (got[~seen] == 0).all()
    assert (np.abs(glse[seen] - wlse[seen]) <= e[seen] + 2.0 ** -20 * (1 + np.abs(wlse[seen]))).all()


# binary16 results span 2^-24 .. 2^16: scales there are fewer apart
FAR = {"bf16": (1e-9, 1e9), "f16": (1e-2, 300.0)}


def rising(dtype):
    lo, hi = FAR[dtype]
    return lambda n: lo * (hi / lo) ** (np.arange(n) / max(1, n - 1))


# few rows; many rows, tiles widened on the way; widened ahead (1024 rows and
# more); each also split over the cache, and sequences in parts
FORMS = [([2, 1], [500, 400], 4, 2), ([5, 1], [300, 130], 6, 1), ([100, 70], [500, 333], 4, 2),
         ([300, 20], [300, 200], 8, 2), ([1], [5000], 4, 1), ([40], [3000], 2, 1), ([257], [2100], 8, 1),
         ([1] * 12, [4500] + [300] * 11, 4, 1)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q,kv,Hq,H", FORMS)
def test_rising_scales(qg, dtype, D, q, kv, Hq, H):
    """Scales that grow along the sequence: early rows do not see the large ones."""
    check(qg, q, kv, Hq, H, D, 16, dtype, rising(dtype))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("q,kv,Hq,H", FORMS)
def test_falling_scales(qg, dtype, q, kv, Hq, H):
    check(qg, q, kv, Hq, H, 128, 32, dtype, lambda n: rising(dtype)(n)[::-1], causal=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q,kv,Hq,H", FORMS)
def test_large_scales_that_hardly_weigh(qg, dtype, D, q, kv, Hq, H):
    """Every other block has a value scale far above and a weight of about
    e^-40: the result is the others'."""
    big = {"bf16": 2.0 ** 30, "f16": 2.0 ** 14}[dtype]
    check(qg, q, kv, Hq, H, D, 16, dtype, lambda n: np.where(np.arange(n) % 2, 0.03 * big, 0.03),
          quiet=lambda i, n: i % 2 == 1)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q,kv,Hq,H", FORMS)
def test_zero_blocks_first(qg, dtype, D, q, kv, Hq, H):
    """Blocks of zeros (scale 0) before the others: whole tiles in which no
    value scale has been met yet, whose tokens the sum still counts."""
    check(qg, q, kv, Hq, H, D, 16, dtype, lambda n: np.where(np.arange(n) < n * 2 // 3, 0, 0.03))
    check(qg, q, kv, Hq, H, D, 16, dtype, lambda n: np.where(np.arange(n) % 5, 0, 0.03))



# few rows, many, and many of ready-made tiles
@pytest.mark.parametrize("q,kv,Hq,H", [([9], [120], 1, 1), ([25], [200], 1, 1), ([16], [150], 2, 1),
                                       ([200], [200], 2, 2), ([150], [330], 1, 1), ([1100], [1100], 1, 1)])
def test_steep_scales(qg, q, kv, Hq, H):
    """Each block's scale 2^12 times the last one's: the new tokens of a wave end
    in different blocks, and hidden tokens beside theirs have scales far above."""
    for bs in (16, 32):
        check(qg, q, kv, Hq, H, 128, bs, "bf16", lambda n: 2.0 ** np.minimum(12.0 * np.arange(n) - 60, 95))


def test_scales_at_the_ends_of_their_range(qg):
    """2^-100 to 2^100, what a cache may hold."""
    for q, kv, Hq, H in FORMS:
        check(qg, q, kv, Hq, H, 64, 16, "bf16", lambda n: 2.0 ** np.linspace(-100, 100, n))
        check(qg, q, kv, Hq, H, 64, 16, "bf16", lambda n: 2.0 ** np.linspace(100, -100, n), causal=False)


def test_a_prompt_among_decoding_steps(qg):
    """A prompt whose tiles are not widened ahead, for the room that the others
    would take, beside sequences of the few-row kernel."""
    for q, kv in (([1100] + [1] * 60, [1100] + [70 + 9 * i for i in range(60)]),
                  ([1] * 30 + [600, 600], [1 + 19 * i for i in range(30)] + [600, 1190])):
        check(qg, q, kv, 4, 2, 128, 32, "bf16", lambda n: np.full(n, 0.03))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("n,L,Hq,H,D", [(16, 100, 2, 2, 128), (20, 90, 1, 1, 64), (60, 150, 4, 2, 128),
                                        (300, 300, 4, 1, 64), (1100, 1100, 1, 1, 128), (40, 2100, 2, 1, 256)])
def test_hidden_tokens_have_no_part(qg, dtype, n, L, Hq, H, D):
    """Other codes and scales in the blocks that a new token does not see leave
    its bits alone."""
    rng = np.random.default_rng(9)
    bs, blocks = 16, -(-L // 16)
    cache = as_cache(qg, make_cache(rng, blocks, H, bs, D))
    table = dev(np.arange(blocks, dtype=np.int32)[None])
    q = torch.from_numpy(rng.normal(size=(n, Hq, D))).to(DTYPES[dtype]).cuda()
    args = (table, dev(np.array([0, n], np.int32)), dev(np.array([L], np.int32)), n, L)
    print(f"hidden tokens {n} of {L}, {Hq}/{H} heads of {D} {dtype}", flush=True)
    first = qg.qattn_kv8(q, cache, *args, return_lse=True)
    cut = L - n // 2  # tokens from here on are others
    b0 = -(-cut // bs)
    sees = b0 * bs - (L - n)  # new tokens that see only blocks before b0
    assert 0 < sees < n
    for scale in (2.0 ** 60, 0.0):
        for t in cache[:2]:
            t[b0:] = torch.randint(-127, 128, t[b0:].shape, dtype=torch.int8, device="cuda") if scale else 0
        for t in cache[2:]:
            t[b0:] = scale
        again = qg.qattn_kv8(q, cache, *args, return_lse=True)
        assert torch.equal(first[0][:sees], again[0][:sees]) and torch.equal(first[1][:sees], again[1][:sees])
