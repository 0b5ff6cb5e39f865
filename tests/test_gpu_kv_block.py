"""The operators together: an attention block whose weights, activations and
cache are IF4, prompts in chunks and then single tokens."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 3)])
def test_chunks_do_not_matter(window, sinks):
    # the cache's bytes are the same however a prompt is cut, and outputs differ by
    # roundings only: attention's to bf16 (2^-9), which the second product's
    # 4-bit operand can turn into a neighbouring code -- a step of a sixth of a
    # group's largest value -- for the few values next to a boundary
    from adaptive_block_scaled_amd import decoder_attention as da
    prompts, got, caches = [130, 37, 1], [], []
    for chunk in (130, 64, 7):
        block = da.random_block(256, 8, 2, 64, 16, 16, window, sinks)
        _, outs, _, _ = da.serve(block, prompts, 3, chunk, 256)
        got.append(outs)
        caches.append([block.pages.owned[i] for i in range(3)])
        bytes_ = [t.clone() for t in block.cache]
        rows = [[t[block.pages.owned[i]][:prompts[i] // 16] for t in bytes_] for i in range(3)]
        if len(got) > 1:
            for a, b in zip(rows, first):
                for x, y in zip(a, b):
                    assert torch.equal(x, y)
        else:
            first = rows
    for outs in got[1:]:
        for a, b in zip(outs, got[0]):
            assert a.shape == b.shape
            assert float((a - b).norm() / b.norm()) < 0.03


def test_close_to_an_unquantized_cache():
    # IF4 keeps normal values within about a tenth (4.5 bits per value): an
    # output that averages many of them is nearer than that
    from adaptive_block_scaled_amd import decoder_attention as da
    block = da.random_block(512, 8, 4, 128, 40, 64)
    xs, outs, _, _ = da.serve(block, [300, 90], 5, 100, 512)
    for x, out in zip(xs, outs):
        want = block.reference(x)
        assert float((out - want).norm() / want.norm()) < 0.25


def test_pages_are_given_and_taken_back():
    from adaptive_block_scaled_amd import decoder_attention as da
    pages = da.Pages(3, 16, "cuda")
    a, b = pages.extend("a", 17), pages.extend("b", 16)
    assert len(set(a + b)) == 33 and len(pages.free) == 0
    with pytest.raises(MemoryError):
        pages.extend("b", 1)
    pages.release("a")
    assert len(pages.extend("b", 1)) == 1
