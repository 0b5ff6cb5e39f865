"""How much workspace attention over the KV cache asks for: sizes only, no GPU."""
import os

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
