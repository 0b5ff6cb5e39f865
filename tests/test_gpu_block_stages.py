"""The operators as a decoder's attention block runs them: projections in FP8, norm and
rotation, the IF4 cache and attention, weights summed, eviction, and the next tokens."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def block(da, precision="fp8", rotary=64, weights_of=0, pages=60, page_size=16, **kw):
    return da.random_block(256, 8, 2, 64, pages, page_size, rotary=rotary, positions=400, precision=precision,
                           weights_of=weights_of, **kw)


@pytest.mark.parametrize("precision", ["if4", "fp8"])
@pytest.mark.parametrize("rotary", [0, 32, 64])
def test_close_to_an_unquantized_cache(precision, rotary):
    # IF4 keeps normal values within about a tenth: an output that averages many is nearer
    from adaptive_block_scaled_amd import decoder_attention as da
    b = block(da, precision, rotary)
    xs, outs, _, _ = da.serve(b, [150, 33], 4, 64, 256)
    for x, out in zip(xs, outs):
        want = b.reference(x)
        assert out.shape == want.shape and float((out - want).norm() / want.norm()) < 0.25


def test_chunks_do_not_matter():
    # the cache's bytes are the same however a prompt is cut: a token's projection, norm and
    # rotation do not depend on its neighbours (the product's tile may, whose sums are then in
    # another order: bf16 projections, one of 2^8 steps apart now and then)
    from adaptive_block_scaled_amd import decoder_attention as da
    outs = []
    for chunk in (130, 64, 7):
        _, o, _, _ = da.serve(block(da), [130, 37, 1], 3, chunk, 256)
        outs.append(o)
    for other in outs[1:]:
        for a, c in zip(other, outs[0]):
            assert a.shape == c.shape and float((a - c).norm() / c.norm()) < 0.03


def test_weights_of_every_row_add_up_to_one():
    """Every row's weights add up to one per query head, whatever the cut."""
    from adaptive_block_scaled_amd import decoder_attention as da
    b = block(da, weights_of=200)
    da.serve(b, [130, 37], 3, 50, 256)
    for s, n in ((0, 133), (1, 40)):
        row = b.mass[b.mass_row[s]]
        # 4 query heads of each kv head; the first tokens of a chunk start from nothing, so
        # that every row is counted once
        assert bool((row[:, :n].double().sum(1) - 4 * n).abs().max() < 4 * n * 1e-5)
        assert not bool(row[:, n:].any())


def test_eviction_that_keeps_all_changes_nothing():
    from adaptive_block_scaled_amd import decoder_attention as da
    a, b = block(da), block(da, weights_of=400)
    _, want, _, _ = da.serve(a, [120, 45], 4, 64, 256)
    _, got, _, _ = da.serve(b, [120, 45], 4, 64, 256, keep=120)
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_eviction_keeps_the_tokens_that_matter():
    """After the cut a decode step is attention over what was kept: the same as with those
    tokens' keys and values read back, and the pages are given and taken as counted."""
    from adaptive_block_scaled_amd import decoder_attention as da, kv_cache
    b = block(da, weights_of=400, pages=40)
    prompts, keep = [200, 90, 40], 64
    xs, _, _, _ = da.serve(b, prompts, 0, 64, 256)
    mass = b.mass.clone()
    lens = dict(b.pages.lens)
    with pytest.raises(MemoryError):
        held = [b.pages.free.pop() for _ in range(len(b.pages.free) - 3)]
        try:
            b.evict([0, 1, 2], keep, recent=8, sinks=2)
        finally:
            b.pages.free += held
    assert b.pages.lens == lens and torch.equal(b.mass, mass)
    free = len(b.pages.free)
    b.evict([0, 1, 2], keep, recent=8, sinks=2)
    assert [b.pages.lens[s] for s in range(3)] == [64, 64, 40]
    assert len(b.pages.free) == free + 13 + 6 - 4 - 4 and b.pages.seen == {0: 200, 1: 90, 2: 40}
    owned = sum((b.pages.owned[s] for s in range(3)), [])
    assert len(set(owned + b.pages.free)) == 40
    # the kept tokens' sums are the largest ones, in the order of the tokens
    for s, n in ((0, 200), (1, 90)):
        for h in range(2):
            old = mass[b.mass_row[s], h, :n]
            want = sorted(list(range(2)) + list(range(n - 8, n)) +
                          (old[2:n - 8].argsort(descending=True, stable=True)[:keep - 10] + 2).tolist())
            assert torch.equal(b.mass[b.mass_row[s], h, :keep], old[want])
    # a decode step: the block's attention against one over the values read back
    got = b.forward(torch.cat([xs[s][-1:] for s in range(3)]), [0, 1, 2], [1, 1, 1])
    for s in range(3):
        n = b.pages.lens[s]
        slots = torch.tensor([b.pages.owned[s][j // 16] * 16 + j % 16 for j in range(n)], device="cuda")
        k, v = (t.float() for t in kv_cache.read(b.cache, slots, **b.exps))
        pos = torch.tensor([b.pages.seen[s] - 1], device="cuda")
        q = b._project(xs[s][-1:], -8, pos)[0].float()
        p = torch.softmax(torch.einsum("hd,nhd->hn", q[0], k.repeat_interleave(4, 1)) * 64 ** -0.5, 1)
        o = torch.einsum("hn,nhd->hd", p, v.repeat_interleave(4, 1)).bfloat16()
        want = b._linear(o.reshape(1, -1), b.w_o, -8)
        # attention's own roundings (2^-8 of bf16, 2^-10 of its operands), then FP8's step of
        # 2^-3 where one of them turns a code of 3 bits into its neighbour
        assert float((got[s] - want[0]).norm() / want.norm()) < 0.02


@pytest.mark.parametrize("free", [4, 5, 8])
def test_eviction_from_a_full_cache(free):
    """Free pages for one sequence's kept tokens are enough for any number of sequences, and
    the outcome is that of an eviction with room for all at once."""
    from adaptive_block_scaled_amd import decoder_attention as da, kv_cache
    prompts, keep = [200, 70, 90, 66], 64  # of pages of 16: 4 each are kept
    roomy, full = block(da, weights_of=400, pages=60), block(da, weights_of=400, pages=60)
    for b in (roomy, full):
        da.serve(b, prompts, 0, 64, 256)
    held = [full.pages.free.pop() for _ in range(len(full.pages.free) - free)]
    for b in (roomy, full):
        b.evict(range(4), keep, recent=8, sinks=2)
    assert full.pages.lens == roomy.pages.lens == {s: 64 for s in range(4)}
    owned = sum((full.pages.owned[s] for s in range(4)), [])
    assert sorted(owned + full.pages.free + held) == list(range(60))
    assert torch.equal(full.mass, roomy.mass)
    for s in range(4):
        kv = [kv_cache.read(b.cache, torch.tensor([b.pages.owned[s][j // 16] * 16 + j % 16 for j in range(64)],
                                                  device="cuda"), **b.exps) for b in (full, roomy)]
        assert all(torch.equal(x, y) for x, y in zip(*kv))


def test_an_eviction_that_fails_takes_no_pages(monkeypatch):
    # no memory for the choice of tokens: the block is as before, and the same call goes through later
    from adaptive_block_scaled_amd import decoder_attention as da
    b = block(da, weights_of=100)
    b.forward(torch.randn(50, 256, device="cuda").bfloat16(), ["a"], [50])
    before = (list(b.pages.free), {s: list(p) for s, p in b.pages.owned.items()}, dict(b.pages.lens), b.mass.clone())

    def none(*a, **kw):
        raise torch.OutOfMemoryError("none left")
    for owner, name in ((da.kv_evict, "select"), (b.pages, "rows")):
        with monkeypatch.context() as m:
            calls = [getattr(owner, name)]
            # (the first table is that of the pages the sequence has)
            m.setattr(owner, name, none if name == "select" else lambda p: calls.pop()(p) if calls else none())
            with pytest.raises(torch.OutOfMemoryError):
                b.evict(["a"], 20, recent=4)
        assert (b.pages.free, b.pages.owned, b.pages.lens) == before[:3] and torch.equal(b.mass, before[3])
    b.evict(["a"], 20, recent=4)
    assert b.pages.lens == {"a": 20} and len(b.pages.owned["a"]) == 2


def test_sums_of_released_sequences_are_used_again():
    from adaptive_block_scaled_amd import decoder_attention as da
    b = block(da, weights_of=100, pages=60)
    xs = torch.randn(30, 256, device="cuda").bfloat16()
    for s in range(20):
        b.forward(xs, [s], [30])
    rows = len(b.mass)
    for s in range(20):
        b.release(s)
    b.forward(xs, ["next"], [30])
    assert len(b.mass) == rows and float((b.mass[b.mass_row["next"]].double().sum(1) - 120).abs().max()) < 1e-2
    with pytest.raises(ValueError, match="tokens that weights"):
        b.forward(torch.cat([xs] * 3), ["next"], [90])
    assert b.pages.lens["next"] == 30


def test_refusals():
    from adaptive_block_scaled_amd import decoder_attention as da
    with pytest.raises(ValueError, match="precision"):
        block(da, "bf16")
    with pytest.raises(ValueError, match="window"):
        block(da, weights_of=10, window=16)
    b = block(da)
    b.forward(torch.zeros(3, 256, device="cuda").bfloat16(), ["a"], [3])
    with pytest.raises(ValueError, match="weights"):
        b.evict(["a"], 2)
    with pytest.raises(ValueError, match="table"):
        b.forward(torch.zeros(398, 256, device="cuda").bfloat16(), ["a"], [398])
    with pytest.raises((ValueError, RuntimeError)):
        b.forward(torch.zeros(2, 250, device="cuda").bfloat16(), ["a"], [2])
    assert b.pages.lens == {"a": 3} and b.pages.seen == {"a": 3}
    b = block(da, weights_of=10)
    b.forward(torch.zeros(6, 256, device="cuda").bfloat16(), ["a"], [6])
    owned, free = dict(b.pages.owned), list(b.pages.free)
    for args, kw in (((["a"], 0), {}), ((["a"], 2), dict(recent=2, sinks=1)), ((["a"], 2), dict(sinks=-1)),
                     ((["a", "a"], 2), {})):
        with pytest.raises(ValueError, match="keep|twice"):
            b.evict(*args, **kw)
    assert b.pages.owned == owned and b.pages.free == free and b.pages.lens == {"a": 6}


def test_command(capsys):
    from adaptive_block_scaled_amd import decoder_attention as da
    da.main("--hidden 256 --heads 4 --kv-heads 2 --dim 64 --batch 3 --prompt 300 --chunk 128 --steps 2 "
            "--precision fp8 --rotary 64 --keep 64".split())
    assert "decode_ms_per_step" in capsys.readouterr().out
