"""Attention over the KV cache in batches of more sequences than a wave has lanes
(workgroups count a ragged batch 64 sequences at a time), with starts, lengths and pages
out of order, and at the lower edge of a window."""
import numpy as np
import pytest

from test_gpu_kv_attention import Batch, kvc  # noqa: F401  (kvc: the module's fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KEPT = 0x4321  # bf16 bits that no row of these calls can get


def ragged(batch, chunks, longest):
    """(lengths, chunks) of `batch` sequences, some of them without rows or keys."""
    c = [chunks[i * 7 % len(chunks)] for i in range(batch)]
    return [0 if i % 31 == 5 else max(n, (i * 37) % 90 + 1) if i % 29 else longest for i, n in enumerate(c)], c


@pytest.mark.parametrize("batch", [64, 65, 128, 129, 150])
@pytest.mark.parametrize("heads,kv_heads,dim,chunks", [
    (8, 2, 64, [1, 0, 5, 16, 2, 3, 30, 1, 0, 9]),        # 33 to 128 rows
    (8, 1, 128, [1, 0, 3, 16, 2, 1, 11, 0, 7]),
    (7, 1, 128, [1, 0, 30, 2, 3, 0, 19, 1, 40, 1, 1]),   # prompts
    (4, 2, 64, [1, 70, 2, 0, 33, 1, 1, 5]),
    (5, 1, 256, [1, 0, 30, 2, 3, 0, 9, 1, 1]),           # wide heads
])
def test_ragged_batches(kvc, batch, heads, kv_heads, dim, chunks):
    lens, c = ragged(batch, chunks, 400)
    b = Batch(kvc, lens, c, heads, kv_heads, dim, 16, 31)
    want = [b.check(kvc, max_len=n) for n in (1, 400, 6000)]
    assert all(w.shape == want[0].shape for w in want)
    b.check(kvc, window=33, sinks=2, max_len=400)


@pytest.mark.parametrize("batch,at", [(65, 0), (65, 64), (128, 63), (150, 70), (150, 149)])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (16, 2, 128), (6, 1, 256)])
def test_many_single_tokens_beside_a_long_chunk(kvc, batch, at, heads, kv_heads, dim):
    # the chunk first, last, and at the borders of the groups of 64
    lens, c = ragged(batch, [1, 1, 0, 1, 2, 1, 1], 300)
    lens[at], c[at] = 500, 120
    b = Batch(kvc, lens, c, heads, kv_heads, dim, 16, 32)
    for max_len in (64, 500, 9000):
        b.check(kvc, max_len=max_len)


@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 64), (40, 1, 128), (60, 1, 128), (16, 1, 256)])
def test_indices_out_of_range_are_the_nearest_ones(kvc, heads, kv_heads, dim):
    b = Batch(kvc, [40, 50], [3, 5], heads, kv_heads, dim, 16, 33)
    table, lens, starts = b.device()
    q = b.q.cuda()

    def bits(table=table, lens=lens, starts=starts, **kw):
        out = torch.full(q.shape, KEPT, dtype=torch.int16, device="cuda").view(torch.bfloat16)
        i32 = dict(dtype=torch.int32, device="cuda")
        kw = {**dict(max_q=5, max_len=1), **b.exps, **kw}
        return kvc.attention(q, b.cache, table, torch.as_tensor(lens, **i32), torch.as_tensor(starts, **i32),
                             out=out, **kw).view(torch.int16)

    wild, held = table.clone(), table.clone()
    wild[0, 1], wild[1, 2], wild[1, 0] = 1 << 30, -(1 << 31), b.cache.k_codes.shape[0]
    held[0, 1], held[1, 2], held[1, 0] = b.cache.k_codes.shape[0] - 1, 0, b.cache.k_codes.shape[0] - 1
    for max_len in (1, 100000):
        kw = dict(max_len=max_len)
        assert torch.equal(bits(table=wild, **kw), bits(table=held, **kw))
        plain = bits(**kw)
        assert torch.equal(bits(starts=[0, 3, 1 << 30], **kw), plain)
        assert torch.equal(bits(starts=[-5, 3, 8], **kw), plain)
        assert torch.equal(bits(starts=[-(1 << 31), 3, (1 << 31) - 1], **kw), plain)
        assert bool((bits(lens=[-40, -(1 << 31)], **kw) == 0).all())
    # starts that descend: the first sequence has no rows, the second those from 2 on
    got = bits(starts=[4, 2, 7])
    assert torch.equal(got[2:7], bits(starts=[2, 2, 7])[2:7])
    assert bool((got[:2] == KEPT).all()) and bool((got[7:] == KEPT).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,chunk", [(2, 1), (16, 1), (16, 3), (8, 150)])
@pytest.mark.parametrize("window", [1, 31, 64, 97, 200])
def test_the_lower_edge_of_a_window(kvc, dim, heads, chunk, window):
    # a NaN in K of one key and in V of another: the rows that see them, and no others, have it.
    # Both slide out of the window within the chunk, or between two calls of a single token
    for shift in range(2 if chunk < 4 else 1):
        n = 401 - shift

        def edit(b, k, v):
            last = 401 - chunk + (0 if chunk < 4 else 70)  # the position of the first row that sees neither
            k[last - window, 0, 7] = float("nan")
            v[last - window - (5 if chunk > 4 else 0), 1, dim - 1] = float("nan")
        b = Batch(kvc, [n], [chunk], heads, 2, dim, 16, 34, edit=edit)
        for max_len in (1, n):
            got = b.check(kvc, window=window, max_len=max_len)
            rows = np.isnan(got).any((1, 2))
            assert rows.any() == (shift == 1 or chunk > 4) and (chunk == 1 or not rows[-1])


@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 64), (8, 2, 64), (40, 1, 128), (6, 1, 256)])
def test_a_hint_of_no_keys(kvc, heads, kv_heads, dim):
    # max_len = 0 is in order (only the speed depends on it), also by default, where the
    # page table has no room; chunks that differ, so that workgroups count what there is
    for chunks in ([1, 1, 1], [70, 1, 0, 3, 1, 1], [1, 1, 1, 1, 1, 1, 1, 90, 1]):
        lens = [300, 40, 0, 7, 64, 1, 33, 200, 5][:len(chunks)]
        b = Batch(kvc, lens, chunks, heads, kv_heads, dim, 16, 35)
        b.check(kvc, max_len=0)
        table, seq_lens, starts = b.device()
        out = kvc.attention(b.q.cuda(), b.cache, table[:, :0].contiguous(), seq_lens, starts, max_q=max(chunks), **b.exps)
        assert bool((out == 0).all())


def test_one_workspace_serves_a_batch_that_shrinks(kvc):
    # sized once for the most; of these, 40 sequences fill the chip without splits and the
    # fewer the more splits
    b = Batch(kvc, [600 - i for i in range(40)], [1] * 40, 8, 8, 128, 16, 36)
    table, lens, starts = b.device()
    q = b.q.cuda()
    need = kvc.workspace_bytes(b.cache, total_q=40, heads=8, batch=40, max_q=1, max_len=600)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = b.check(kvc, max_len=600)
    for n in (40, 30, 11, 4, 1):
        kw = dict(max_q=1, max_len=600, **b.exps)
        got = kvc.attention(q[:n], b.cache, table[:n], lens[:n], starts[:n + 1], workspace=ws, **kw)
        assert torch.equal(got, kvc.attention(q[:n], b.cache, table[:n], lens[:n], starts[:n + 1], **kw))
        # (other splits: the rounding to bf16 and the arithmetic within, of values below 4)
        assert np.abs(got.cpu().double().numpy() - want[:n]).max() < 2.0 ** -5


@pytest.mark.parametrize("heads,kv_heads,dim,chunks", [
    (8, 1, 64, [16, 3, 11]), (8, 1, 128, [16, 3, 11]), (8, 2, 128, [150, 3, 90]), (8, 2, 64, [150, 3, 90]),
    (6, 1, 256, [40, 3, 90]), (16, 2, 128, [1, 1, 1, 1, 2, 1, 1, 120, 1]),
])
def test_chunks_in_a_graph(kvc, heads, kv_heads, dim, chunks):
    # every kernel and the join, replayed with other queries and lengths between eager calls
    lens = [2100, 700, 900, 1, 64, 333, 40, 1700, 500][:len(chunks)]
    b = Batch(kvc, lens, chunks, heads, kv_heads, dim, 16, 37)
    table, seq_lens, starts = b.device()
    q = b.q.cuda()
    out = torch.empty_like(q)
    sizes = dict(max_q=max(chunks), max_len=2100)
    need = kvc.workspace_bytes(b.cache, total_q=len(q), heads=heads, batch=len(lens), **sizes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step(out):
        return kvc.attention(q, b.cache, table, seq_lens, starts, out=out, workspace=ws, **sizes, **b.exps)

    step(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(out)
    for i in range(4):
        q.copy_(torch.randn_like(q.float()).bfloat16())
        seq_lens.copy_((seq_lens - 1).clamp(min=0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), step(torch.empty_like(q)).view(torch.int16)), i
        torch.cuda.synchronize()
