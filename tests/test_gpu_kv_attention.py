"""Attention over the paged IF4 KV cache against a plain 64-bit form, element
by element within the bound that the operator's stated arithmetic allows
(tests/kv_reference.py derives it)."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvc():
    from adaptive_block_scaled_amd import kv_cache
    return kv_cache


class Batch:
    """A batch of sequences in a cache whose other bytes are random (NaN scale
    bytes among them): lens[b] keys, chunks[b] rows of q."""

    def __init__(self, kvc, lens, chunks, heads, kv_heads, dim, page, seed=0, k_exp=-6, v_exp=-8,
                 edit=None, gain=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lens), max(need + [1]) + 1), -7, np.int32)  # padding: no page
        self.cache = kvc.empty(pages, page, kv_heads, dim)
        for t in self.cache:
            t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
        first = 0
        for b, n in enumerate(lens):
            self.table[b, :need[b]] = order[first:first + need[b]]
            first += need[b]
            if n == 0:
                continue
            k = torch.randn(n, kv_heads, dim, generator=g) * gain
            v = torch.randn(n, kv_heads, dim, generator=g)
            k[:, :, 3] *= 6.0
            if edit:
                edit(b, k, v)
            j = np.arange(n)
            slots = self.table[b, j // page].astype(np.int64) * page + j % page
            kvc.append(self.cache, k.bfloat16().cuda(), v.bfloat16().cuda(),
                       torch.from_numpy(slots).cuda(), k_exp, v_exp)
        self.lens, self.starts = list(lens), np.concatenate([[0], np.cumsum(chunks)])
        self.max_q = max(chunks)
        self.exps = dict(k_exp=k_exp, v_exp=v_exp)
        self.q = torch.randn(int(self.starts[-1]), heads, dim, generator=g).bfloat16()
        self.page = page

    def device(self):
        i32 = dict(dtype=torch.int32, device="cuda")
        return (torch.tensor(self.table, **i32), torch.tensor(self.lens, **i32),
                torch.tensor(self.starts, **i32))

    def run(self, kvc, q=None, **kw):
        kw.setdefault("max_q", self.max_q)
        return kvc.attention(self.q.cuda() if q is None else q, self.cache, *self.device(),
                             **self.exps, **kw)

    def reference(self, scale=None, **kw):
        cache = {n: t.cpu().numpy() for n, t in self.cache._asdict().items()}
        scale = self.q.shape[-1] ** -0.5 if scale is None else scale
        kw.pop("max_len", None)
        return ref.attention(self.q.double().numpy(), cache, self.table, self.lens, self.starts,
                             scale, **self.exps, **kw)

    def check(self, kvc, **kw):
        got = self.run(kvc, **kw).cpu().double().numpy()
        want, bound = self.reference(**kw)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        fine = ~np.isnan(want)
        over = (np.abs(got - want) - bound)[fine]
        assert over.size == 0 or over.max() <= 0.0, over.max()
        return got


LAYOUTS = [  # heads, kv_heads, dim, page
    (1, 1, 128, 16), (8, 8, 64, 16), (16, 2, 128, 64), (21, 3, 256, 16), (14, 2, 64, 48),
    (32, 1, 128, 32), (6, 2, 256, 128), (8, 1, 128, 16),
]


@pytest.mark.parametrize("heads,kv_heads,dim,page", LAYOUTS)
def test_single_tokens(kvc, heads, kv_heads, dim, page):
    Batch(kvc, [1, 2, 15, 16, 17, 31, 33, 64, 100, 257], [1] * 10, heads, kv_heads, dim, page).check(kvc)


@pytest.mark.parametrize("heads,kv_heads,dim,page", LAYOUTS)
def test_ragged_chunks(kvc, heads, kv_heads, dim, page):
    # a chunk alone, chunks over a context, single tokens, no rows at all
    Batch(kvc, [5, 40, 33, 130, 64, 9], [5, 17, 1, 70, 0, 2], heads, kv_heads, dim, page, 1).check(kvc)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (32, 1), (40, 33), (64, 0), (1000, 4), (5, 500)])
def test_window_and_sinks(kvc, dim, window, sinks):
    Batch(kvc, [150, 300, 31], [40, 3, 31], 4, 2, dim, 16, 2).check(kvc, window=window, sinks=sinks)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing(kvc, dim):
    # no keys at all, and more rows than keys: positions before the first key
    b = Batch(kvc, [0, 3, 0, 20], [4, 9, 1, 25], 8, 2, dim, 16, 3)
    got = b.check(kvc)
    assert (got[:4] == 0).all() and (got[4:10] == 0).all() and (got[13] == 0).all()
    b.check(kvc, window=2, sinks=1)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_not_causal(kvc, dim):
    Batch(kvc, [33, 100, 0], [7, 40, 3], 6, 3, dim, 32, 4).check(kvc, causal=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("chunks", [[1, 1], [40, 130]])
def test_nan_of_keys_that_a_row_does_not_see(kvc, dim, chunks):
    # the oldest tokens slide out of the window, the newest are hidden from
    # earlier rows; a row that sees one is NaN in the dims that it touches
    def edit(b, k, v):
        k[len(k) - 1, 0, 5] = float("inf")
        v[len(v) - 2, 1, 40] = float("nan")
        v[2, 0, 0] = float("-inf")
        k[3, 1, 63] = float("nan")
    b = Batch(kvc, [150, 300], chunks, 8, 2, dim, 16, 5, edit=edit)
    for kw in (dict(window=20), dict(window=20, sinks=2), dict(window=20, sinks=3), dict()):
        got = b.check(kvc, **kw)
        assert np.isnan(got).any() and (not kw or not np.isnan(got).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_not_finite_queries(kvc, dim):
    b = Batch(kvc, [50, 200], [3, 90], 4, 2, dim, 16, 6)
    b.q[1, 2, 7] = float("inf")
    b.q[60, 0, 0] = float("nan")
    got = b.run(kvc).cpu()
    want = torch.zeros(got.shape[:2], dtype=torch.bool)
    want[1, 2] = want[60, 0] = True
    assert torch.equal(torch.isnan(got).all(-1), want) and torch.equal(torch.isnan(got).any(-1), want)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("chunk", [1, 150])
def test_splits_of_the_keys(kvc, dim, chunk):
    # the same call with other hints of the length: other splits, same definition
    b = Batch(kvc, [2100, 700], [chunk, chunk], 8, 1, dim, 64, 7)
    for max_len in (1, 500, 2100, 1 << 20, None):
        b.check(kvc, max_len=max_len)
    b.check(kvc, window=100, sinks=5, max_len=100000)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("chunk", [1, 20, 150])
def test_scores_that_rise_and_fall_along_the_keys(kvc, dim, chunk):
    # the running maximum moves in nearly every step of the first half of the
    # heads' rows, by little or by much, and in none of the others'
    def edit(b, k, v):
        ramp = torch.linspace(-20, 40, len(k))
        k[:, 0, :16] = torch.sign(torch.randn(16, generator=torch.Generator().manual_seed(1))) * ramp[:, None]
        k[:, 1, 16:32] = (ramp.flip(0) ** 3 / 1600)[:, None]
    b = Batch(kvc, [700, 411], [chunk, chunk], 8, 2, dim, 16, 15, k_exp=-4, edit=edit)
    b.check(kvc)
    b.check(kvc, max_len=64)
    b.check(kvc, window=200, sinks=70)


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (7, 1, 128), (6, 1, 256)])
def test_many_lengths_at_once(kvc, heads, kv_heads, dim):
    # decodes and chunks of all sizes in one call: tiles with few rows, with many, none
    lens = [1, 16, 63, 64, 65, 128, 191, 300, 511, 640, 777, 900]
    chunks = [1, 16, 2, 60, 65, 1, 0, 37, 5, 22, 1, 48]
    b = Batch(kvc, lens, chunks, heads, kv_heads, dim, 32, 16)
    for max_len in (None, 900, 6000):
        b.check(kvc, max_len=max_len)
    b.check(kvc, window=65, sinks=1)


@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 64), (24, 1, 64), (16, 2, 128), (6, 1, 256), (40, 1, 128)])
def test_single_tokens_beside_a_long_chunk(kvc, heads, kv_heads, dim):
    # most sequences bring one token or two, some none, one a chunk that is far longer
    lens = [700, 33, 1, 400, 257, 64, 900, 5, 650, 310, 12, 800]
    chunks = [1, 1, 1, 150, 1, 2, 1, 0, 1, 17, 1, 3]
    b = Batch(kvc, lens, chunks, heads, kv_heads, dim, 16, 17)
    for max_len in (None, 64, 900, 9000):
        b.check(kvc, max_len=max_len)
    b.check(kvc, window=100, sinks=3)
    got = [b.run(kvc) for _ in range(3)]
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


@pytest.mark.parametrize("chunk", [1, 33])
def test_large_scores_and_scales(kvc, chunk):
    # sharp softmax (one key takes nearly all), tiny and huge q, scale 0
    for gain, scale in ((8.0, None), (1.0, 0.0), (1.0, 3e-5), (1.0, 0.5)):
        Batch(kvc, [300], [chunk], 4, 2, 128, 16, 8, gain=gain).check(kvc, scale=scale)
    b = Batch(kvc, [200], [chunk], 4, 2, 128, 16, 9)
    b.q = (b.q.float() * 2.0 ** 40).bfloat16()
    b.check(kvc, scale=2.0 ** -44)
    b.q[0, 1] = 0.0
    b.q[:, 2] = (b.q[:, 2].float() * 2.0 ** -100).bfloat16()
    b.check(kvc, scale=2.0 ** -44)


@pytest.mark.parametrize("chunk", [1, 200])
def test_strides_streams_and_repeats(kvc, chunk):
    b = Batch(kvc, [400, 300], [chunk, chunk], 8, 2, 128, 32, 10)
    want = b.run(kvc)
    total = want.shape[0]
    fused = torch.full((total, 12, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    fused[:, :8] = b.q.cuda()
    held = torch.full((10, total, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    need = kvc.workspace_bytes(b.cache, total_q=total, heads=8, batch=2, max_q=chunk, max_len=400)
    ws = torch.empty(need + 64, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = b.run(kvc, q=fused[:, :8], out=held[1:9].transpose(0, 1), workspace=ws, max_len=400)
    side.synchronize()
    assert torch.equal(got, b.run(kvc, max_len=400))
    assert bool((held[0] == 5.0).all()) and bool((held[9] == 5.0).all())
    for _ in range(3):
        assert torch.equal(b.run(kvc), want)


def test_in_a_graph(kvc):
    # a decode step's append and attention, replayed while the lengths and the
    # inputs change in place
    b = Batch(kvc, [70, 600, 10], [1, 1, 1], 16, 2, 128, 16, 11)
    table, lens, starts = b.device()
    q = b.q.cuda()
    k = torch.randn(3, 2, 128, device="cuda").bfloat16()
    slots = table.long()[torch.arange(3), (lens.long() - 1) // 16] * 16 + (lens.long() - 1) % 16
    out = torch.empty_like(q)
    need = kvc.workspace_bytes(b.cache, total_q=3, heads=16, batch=3, max_q=1, max_len=600)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

    def step():
        kvc.append(b.cache, k, k, slots, **b.exps)
        kvc.attention(q, b.cache, table, lens, starts, max_q=1, max_len=600, out=out, workspace=ws,
                      **b.exps)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        q.copy_(torch.randn_like(q.float()).bfloat16())
        lens.sub_(1)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out), i


def test_odd_tables_and_starts_stay_inside(kvc):
    # device-side indices out of range are read as the nearest valid ones
    b = Batch(kvc, [40, 50], [3, 2], 4, 2, 64, 16, 12)
    table, lens, starts = b.device()
    kw = dict(max_q=3, **b.exps)
    wild = table.clone()
    wild[0, 1], wild[1, 2] = 1 << 30, -(1 << 31)
    held = table.clone()
    held[0, 1], held[1, 2] = b.cache.k_codes.shape[0] - 1, 0
    q = b.q.cuda()
    assert torch.equal(kvc.attention(q, b.cache, wild, lens, starts, **kw).isnan(),
                       kvc.attention(q, b.cache, held, lens, starts, **kw).isnan())
    full = torch.tensor([table.shape[1] * 16, 50], dtype=torch.int32, device="cuda")
    over = torch.tensor([(1 << 31) - 1, 50], dtype=torch.int32, device="cuda")
    a, c = (kvc.attention(q, b.cache, held, x, starts, **kw) for x in (full, over))
    assert torch.equal(a.view(torch.int16), c.view(torch.int16))
    for s in ([0, 3, 1 << 30], [-5, 3, 5], [4, 2, 5]):
        kvc.attention(q, b.cache, table, lens, torch.tensor(s, dtype=torch.int32, device="cuda"), **kw)
    kvc.attention(q, b.cache, table, -lens, starts, **kw)
    torch.cuda.synchronize()


def test_no_rows_and_no_sequences(kvc):
    b = Batch(kvc, [40], [1], 4, 2, 64, 16, 13)
    table, lens, starts = b.device()
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert kvc.attention(q, b.cache, table, lens, torch.zeros_like(starts), max_q=1).shape == q.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    assert kvc.attention(q, b.cache, torch.empty(0, 3, **i32), torch.empty(0, **i32),
                         torch.zeros(1, **i32), max_q=0).shape == q.shape


def test_refusals_of_the_binding(kvc):
    from adaptive_block_scaled_amd.if4 import IF4Error
    b = Batch(kvc, [40, 700], [3, 2], 4, 2, 64, 16, 14)
    table, lens, starts = b.device()
    q = b.q.cuda()

    def call(match, kind=ValueError, **kw):
        full = dict(q=q, cache=b.cache, page_table=table, seq_lens=lens, q_starts=starts, max_q=3)
        full.update(kw)
        with pytest.raises(kind, match=match):
            kvc.attention(**full)

    call("q must", q=q[0])
    call("q must", q=q.float())
    call("q must", q=q[..., :32])
    call("q must", q=q.cpu())
    call("heads", q=q[:, :3])
    call("page_table", page_table=table[0])
    call("page_table", page_table=table.long())
    call("page_table", page_table=table.t())
    call("seq_lens", seq_lens=lens[:1])
    call("q_starts", q_starts=starts[:2])
    call("q_starts", q_starts=starts.cpu())
    call("scale", scale=-1.0)
    call("scale", scale=float("inf"))
    call("window", window=-1)
    call("window", causal=False, sinks=3)
    call("out must", out=torch.empty(5, 4, 64, device="cuda"))
    call("out must", out=torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda"))
    call("workspace", workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    call("bad shape", kind=IF4Error, max_q=-1)
    call("exponent", kind=IF4Error, k_exp=70)
    call("misaligned", kind=IF4Error,
         q=torch.zeros(5, 4, 68, dtype=torch.bfloat16, device="cuda")[..., :64])
