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


def test_sequences_get_pages_together_or_not_at_all():
    from adaptive_block_scaled_amd.decoder_attention import Pages
    pages = Pages(4, 16, "cpu")
    pages.extend("a", 10)
    before = (dict(pages.lens), {s: list(p) for s, p in pages.owned.items()}, list(pages.free))
    for seqs, counts in ((["a", "b"], [20, 40]), (["b", "a"], [16, 50]), (["a"], [1000])):
        with pytest.raises(MemoryError):
            pages.extend_all(seqs, counts)
        assert (pages.lens, pages.owned, pages.free) == before
    with pytest.raises(ValueError, match="twice"):
        pages.extend_all(["a", "a"], [1, 1])
    slots = pages.extend_all(["a", "b"], [20, 17])
    assert len(slots) == len(set(slots)) == 37 and pages.lens == {"a": 30, "b": 17} and not pages.free
    table, lens = pages.table(["b", "a"])
    assert table.shape == (2, 2) and lens.tolist() == [17, 30]
    flat = [int(table[1, j // 16]) * 16 + j % 16 for j in range(10, 30)] + \
        [int(table[0, j // 16]) * 16 + j % 16 for j in range(17)]
    assert flat == slots


def test_a_block_without_room_forgets_nothing(monkeypatch):
    # the sequences of a call that does not fit keep their lengths: the tokens were not written
    import torch

    from adaptive_block_scaled_amd import decoder_attention as da
    block = da.AttentionBlock.__new__(da.AttentionBlock)
    block.heads, block.kv_heads, block.dim, block.pages = 2, 1, 64, da.Pages(2, 16, "cpu")
    block.w_qkv = ()
    monkeypatch.setattr(da.AttentionBlock, "_linear", staticmethod(lambda x, *w: torch.zeros(len(x), 4 * 64)))
    block.pages.extend("a", 10)
    with pytest.raises(MemoryError):
        block.forward(torch.zeros(24, 8), ["a", "b"], [4, 20])
    assert block.pages.lens == {"a": 10} and len(block.pages.free) == 1
