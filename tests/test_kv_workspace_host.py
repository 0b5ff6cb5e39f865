"""How much workspace attention over the KV cache asks for: sizes only, no GPU."""
import math
import os
import random

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(
    not os.path.exists(os.path.join(ROOT, "adaptive_block_scaled_amd", "libif4.so")), reason="libif4.so not built")


@pytest.fixture(scope="module")
def kvc():
    from adaptive_block_scaled_amd import kv_cache
    return kv_cache


def sizes(kvc, dim=128, heads=64, kv_heads=8, page=64, **kw):
    """(cache, arguments) of a call of these sizes; no pointers."""
    cache = kvc._Cache(pages=1000, page_size=page, kv_heads=kv_heads, head_dim=dim)
    return cache, kvc._Attention(heads=heads, scale=1.0, causal=1, **kw)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_single_tokens_beside_a_long_chunk_have_partial_sums_of_their_own(kvc, dim):
    # (partial sums of all rows of q for each split of the single tokens' keys were 0.5 to 6 GB)
    for singles, chunk, keys in ((8, 2048, 4096), (8, 2048, 131072), (5, 8192, 131072)):
        need = kvc.lib.if4_kv_attention_workspace(*sizes(
            kvc, dim, batch=singles + 1, total_q=singles + chunk, max_q=chunk, max_len=keys))
        assert 0 <= need <= 300e6, (singles, chunk, keys, need)


def test_one_workspace_is_enough_for_all_smaller_calls(kvc):
    # random largest sizes, and calls of every kind within them; it grows with each size
    need, most = kvc.lib.if4_kv_attention_workspace, kvc.lib.if4_kv_attention_workspace_most
    rng, hit = random.Random(5), 0

    def log(hi):
        return min(hi, max(1, round(math.exp(rng.uniform(0, math.log(hi + 1))))))

    for _ in range(1500):
        kv_heads = rng.choice([1, 2, 3, 8])
        heads, dim = kv_heads * rng.choice([1, 2, 4, 7, 8, 16, 24, 40]), rng.choice([64, 128, 256])
        top = dict(batch=log(600), total_q=log(20000), max_q=log(9000), max_len=log(1 << 20))

        def size(f, **kw):
            return f(*sizes(kvc, dim, heads, kv_heads, **kw))
        bound = size(most, **top)
        assert bound <= 280e6
        for name in top:
            assert size(most, **{**top, name: 2 * top[name]}) >= bound
        for _ in range(40):
            call = {n: rng.choice([log(v), v]) for n, v in top.items()}
            if rng.random() < 0.5:
                call["total_q"] = min(call["total_q"], rng.choice([call["batch"], call["batch"] + call["max_q"] - 1]))
            for window, sinks in ((0, 0), (log(1 << 20), rng.choice([0, 64]))):
                n = size(need, window=window, sinks=sinks, **call)
                assert 0 <= n <= bound, (top, call, window, n, bound)
                hit += n > 0
    assert hit > 1000
