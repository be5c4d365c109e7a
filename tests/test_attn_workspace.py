"""What qattn_kv8 asks for as workspace, on the host: it follows the work, not
the batch's size times its longest sequence."""
import random

import pytest


@pytest.fixture(scope="module")
def size():
    from conv_qgemm_amd import qgemm
    return qgemm.lib.qattn_kv8_workspace_size


MB = 1 << 20


def image(tokens, heads, D):
    return -(-tokens // 32) * heads * (4 * 32 * D + 64)


def test_one_prompt_has_its_widened_tiles(size):
    for tokens, Hq, H, D in ((8192, 32, 8, 128), (4096, 32, 8, 64), (131072, 32, 8, 128)):
        assert size(tokens, 1, tokens, tokens, Hq, H, D) == image(tokens, H, D)


@pytest.mark.parametrize("others", [63, 127, 255, 1000])
def test_one_prompt_among_decoding_steps(size, others):
    """Where only one sequence's tiles would be used, no room for all of them."""
    for n in (2048, 8192, 32768):
        assert size(n + others, others + 1, n, n, 32, 8, 128) <= 64 * MB + image(n, 8, 128)


def test_unlike_prompts(size):
    assert size(128 * 9000, 128, 16384, 16384, 32, 8, 128) <= 1024 * MB
    # batches of prompts that use what is asked for keep their widened tiles
    assert size(8 * 1500, 8, 2048, 2048, 32, 8, 128) == 8 * image(2048, 8, 128)
    assert size(16 * 5000, 16, 8192, 8192, 32, 8, 128) == 16 * image(8192, 8, 128)


def test_never_beyond_a_bound(size):
    """Widened tiles up to 1 GB, partial results (at most 2^18 rows of 258
    numbers) beside them."""
    rng = random.Random(3)

    def log(top):
        return int(2 ** rng.uniform(0, top))

    for _ in range(20000):
        D, H = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8, 16])
        seqs, max_q, max_kv = log(12), log(17), log(20)
        tokens = min(seqs * max_q, max_q + log(12) * seqs)
        got = size(tokens, seqs, max_q, max_kv, H * rng.choice([1, 2, 4, 8]), H, D)
        assert got <= 1024 * MB + (1 << 18) * 258 * 4, (tokens, seqs, max_q, max_kv, H, D)
