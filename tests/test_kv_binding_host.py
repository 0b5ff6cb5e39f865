"""Refusals of the KV cache's Python side that need no GPU."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.skipif(
    not os.path.exists(os.path.join(ROOT, "adaptive_block_scaled_amd", "libif4.so")), reason="libif4.so not built")


@pytest.fixture(scope="module")
def kvc():
    from adaptive_block_scaled_amd import kv_cache
    return kv_cache


@pytest.mark.parametrize("kv_heads", [0, -1])
def test_a_cache_has_heads(kvc, kv_heads):
    with pytest.raises(ValueError, match="kv_heads"):
        kvc.empty(2, 16, kv_heads, 64, device="cpu")
