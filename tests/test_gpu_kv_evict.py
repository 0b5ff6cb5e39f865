"""Attention weights added up per cached token against a plain 64-bit form, element by element
within a bound that follows from the operator's stated arithmetic; which tokens stay, and
their bytes in the pages that they move to, exactly."""
import numpy as np
import pytest

import kv_reference as ref
from test_gpu_kv_attention import Batch

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvc():
    from adaptive_block_scaled_amd import kv_cache
    return kv_cache


@pytest.fixture(scope="module")
def ev():
    from adaptive_block_scaled_amd import kv_evict
    return kv_evict


def weights(b, mass, scale, causal=True, window=0, sinks=0, max_q=None):
    """(out, bound).  A score is off by D + 8 roundings of its products and what q's fp16
    leaves out, 2^-24 of the row's largest value each; exp2's argument by 4 roundings of
    its terms; a row's sum by one for each key, a key's sum by one for each row."""
    out, bound = mass.astype(np.float64), np.zeros(mass.shape)
    cache = {n: t.cpu().numpy() for n, t in b.cache._asdict().items()}
    q = b.q.double().numpy()
    heads, dim = q.shape[1:]
    kvh, page = cache["k_codes"].shape[1:3]
    group = heads // kvh
    for i, n in enumerate(b.lens):
        first, t_b = b.starts[i], b.starts[i + 1] - b.starts[i]
        if t_b == 0:
            continue
        n = min(n, b.table.shape[1] * page)
        w = min(n, mass.shape[2])
        out[i, :, max(0, n - t_b):w] = 0
        j = np.arange(n)
        pages, offs = b.table[i, j // page], j % page
        for h in range(kvh):
            k = ref.row_values(cache["k_codes"][pages, h, offs], cache["k_scales"][pages, h, offs], b.exps["k_exp"])
            for r in range(min(t_b, t_b if max_q is None else max_q)):
                pos = n - t_b + r
                seen = np.full(n, True) if not causal else j <= pos
                if window:
                    seen &= (j > pos - window) | (j < sinks)
                if not seen.any():
                    continue
                ks = k[seen]
                for m in range(h * group, (h + 1) * group):
                    x = q[first + r, m]
                    s = (ks @ x) * scale
                    e = np.exp(s - s.max())
                    p = np.zeros(n)
                    p[seen] = e / e.sum()
                    ds = scale * (np.abs(ks) @ np.abs(x) * (dim + 8) * 2.0 ** -24
                                  + 2.0 ** -24 * np.abs(x).max() * np.abs(ks).sum(1)).max()
                    arg = 4 * 2.0 ** -24 * (3 * np.abs(s).max() + 64)
                    rel = np.expm1(2 * ds + arg) + (n + 64) * 2.0 ** -24
                    out[i, h] += np.pad(p, (0, max(0, mass.shape[2] - n)))[:mass.shape[2]]
                    bound[i, h] += np.pad(p, (0, max(0, mass.shape[2] - n)))[:mass.shape[2]] * rel
            bound[i, h] += (np.abs(out[i, h]) * (t_b * group + 4)) * 2.0 ** -24
    return out, bound


def run(kvc, ev, lens, chunks, heads, kv_heads, dim, page, seed=0, width=None, **kw):
    b = Batch(kvc, lens, chunks, heads, kv_heads, dim, page, seed)
    g = np.random.default_rng(seed)
    mass = g.exponential(size=(len(lens), kv_heads, max(lens) + 3 if width is None else width)).astype(np.float32)
    scale = dim ** -0.5
    dev = torch.from_numpy(mass).cuda()
    extra = dict(max_q=b.max_q, max_len=max(lens))
    extra.update(kw)
    got = ev.accumulate(dev, b.q.cuda(), b.cache, *b.device(), scale=scale, k_exp=b.exps["k_exp"], **extra)
    assert got is dev
    mask = {n: kw[n] for n in ("causal", "window", "sinks") if n in kw}
    want, bound = weights(b, mass, scale, max_q=kw.get("max_q"), **mask)
    got = got.cpu().numpy()
    assert (np.abs(got - want) <= bound).all(), np.abs(got - want).max()
    for i, n in enumerate(lens):  # what lies behind a sequence, and a sequence without rows, exactly
        assert np.array_equal(got[i, :, n:], mass[i, :, n:])
        if chunks[i] == 0:
            assert np.array_equal(got[i], mass[i])
    return b, got


CASES = [  # lens, chunks, heads, kv_heads, dim, page
    ([1], [1], 1, 1, 64, 16), ([33], [1], 8, 1, 128, 16), ([300, 17, 1, 64], [1, 1, 1, 1], 8, 2, 128, 32),
    ([500, 90], [1, 1], 12, 4, 256, 64), ([2000], [1], 16, 2, 64, 128), ([40], [40], 2, 2, 64, 16),
    ([130, 61], [70, 61], 4, 1, 128, 64), ([100, 0, 57], [9, 0, 0], 6, 3, 256, 16), ([77, 200], [5, 33], 21, 3, 64, 32),
    ([260], [130], 8, 2, 256, 64), ([390, 390], [129, 1], 10, 2, 128, 16)]


@pytest.mark.parametrize("lens,chunks,heads,kv,dim,page", CASES)
def test_weights(kvc, ev, lens, chunks, heads, kv, dim, page):
    run(kvc, ev, lens, chunks, heads, kv, dim, page, 1)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 0), (20, 3), (64, 64), (1000, 1), (1 << 40, 1 << 40)])
@pytest.mark.parametrize("lens,chunks,dim", [([300], [1], 128), ([410, 200], [150, 33], 64), ([120], [7], 256)])
def test_windows(kvc, ev, lens, chunks, dim, window, sinks):
    run(kvc, ev, lens, chunks, 4, 2, dim, 32, 2, window=window, sinks=sinks)


@pytest.mark.parametrize("lens,chunks,dim", [([90, 31], [33, 2], 64), ([200], [1], 128), ([70], [70], 256)])
def test_all_keys_seen(kvc, ev, lens, chunks, dim):
    run(kvc, ev, lens, chunks, 4, 2, dim, 16, 3, causal=False)


def test_more_rows_than_keys_and_than_max_q(kvc, ev):
    # rows before the first key see nothing; rows past max_q add nothing
    run(kvc, ev, [5, 40], [20, 3], 4, 2, 64, 16, 4)
    run(kvc, ev, [60, 40], [20, 3], 4, 2, 128, 16, 5, max_q=7)


def test_length_hints_change_nothing(kvc, ev):
    for hint in (0, 1, 70, 1 << 20, None):
        run(kvc, ev, [700, 64, 5], [3, 1, 2], 8, 2, 128, 32, 6, max_len=hint)


def test_fewer_sums_than_tokens(kvc, ev):
    run(kvc, ev, [150, 40], [2, 40], 4, 2, 64, 16, 7, width=64)
    run(kvc, ev, [150, 40], [2, 40], 4, 2, 64, 16, 7, width=1)


PARTED = [  # so many rows, and so few blocks of keys, that a block's rows are parted
    ([300, 40], [300, 7], 16, 2, 128, 16), ([700], [200], 8, 1, 64, 32), ([520, 300], [150, 300], 8, 2, 256, 64),
    ([530], [66], 8, 1, 128, 16)]


@pytest.mark.parametrize("kw", [{}, dict(window=20, sinks=3), dict(window=200), dict(causal=False), dict(max_q=70),
                                dict(width=130), dict(max_len=0), dict(max_len=257), dict(max_len=1 << 20)],
                         ids=lambda kw: "-".join("%s_%s" % i for i in kw.items()) or "plain")
@pytest.mark.parametrize("lens,chunks,heads,kv,dim,page", PARTED)
def test_parted_rows(kvc, ev, lens, chunks, heads, kv, dim, page, kw):
    run(kvc, ev, lens, chunks, heads, kv, dim, page, 14, **kw)


NEXT_TO_SINKS = [  # lens, chunks, heads, kv_heads, windows and first tokens
    ([300], [300], 4, 2, [(64, 32), (64, 64), (128, 48), (128, 130), (200, 32), (200, 48), (200, 64)]),
    ([171], [171], 8, 1, [(100, 64), (40, 128)]), ([700], [150], 2, 1, [(512, 64), (512, 130), (600, 40)]),
    ([330, 700, 90], [330, 100, 20], 4, 2, [(250, 64), (600, 48)])]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("lens,chunks,heads,kv,window,sinks", [(*c[:4], *w) for c in NEXT_TO_SINKS for w in c[4]])
def test_windows_that_leave_the_first_tokens(kvc, ev, lens, chunks, heads, kv, dim, window, sinks):
    # rows whose window begins a little behind the first tokens: between the two lie hidden keys,
    # in tiles whose neighbours on both sides are seen whole
    run(kvc, ev, lens, chunks, heads, kv, dim, 16, 21, window=window, sinks=sinks)


def test_weights_of_a_row_sum_to_one(kvc, ev):
    b, got = run(kvc, ev, [3000, 1500], [40, 1], 8, 2, 128, 64, 8)
    mass = torch.zeros(2, 2, 3000, device="cuda")
    ev.accumulate(mass, b.q.cuda(), b.cache, *b.device(), max_q=40, k_exp=b.exps["k_exp"])
    total = mass.double().sum(2).cpu()
    want = torch.tensor([[160.0, 160.0], [4.0, 4.0]], dtype=torch.float64)
    assert bool(((total - want).abs() <= want * 3064 * 2.0 ** -23).all())


def test_hidden_nan_and_seen_nan(kvc, ev):
    # a NaN key is NaN for the rows that see it, and nothing to the others
    b = Batch(kvc, [64], [4], 2, 1, 64, 16, 9)
    k = torch.randn(1, 1, 64).bfloat16().cuda()
    bad = k.clone()
    bad[0, 0, 5] = float("nan")
    slot = torch.tensor([int(b.table[0, 3]) * 16 + 14], device="cuda")  # position 62: rows 2 and 3 see it
    kvc.append(b.cache, bad, k, slot, **b.exps)
    for max_q, nan in ((2, False), (3, True)):
        mass = torch.zeros(1, 1, 64, device="cuda")
        ev.accumulate(mass, b.q.cuda(), b.cache, *b.device(), max_q=max_q, k_exp=b.exps["k_exp"])
        assert bool(mass[0, 0, :63].isnan().all()) == nan and bool(mass.isnan().any()) == nan
        if not nan:
            assert abs(float(mass.double().sum()) - 4) < 1e-5 and not bool(mass[0, 0, 62:].any())


@pytest.mark.parametrize("kw", [{}, dict(window=30, sinks=5), dict(causal=False)], ids=["plain", "window", "full"])
@pytest.mark.parametrize("lens,chunks,heads,kv,dim", [([100], [6], 8, 2, 64), ([90, 40], [16, 3], 2, 1, 128),
                                                      ([200, 70], [120, 5], 4, 2, 64), ([300], [200], 2, 1, 256)])
def test_rows_that_are_nan_reach_what_they_see_only(kvc, ev, lens, chunks, heads, kv, dim, kw):
    b = Batch(kvc, lens, chunks, heads, kv, dim, 16, 22)
    g = np.random.default_rng(22)
    for row, value in ((1, float("nan")), (chunks[0] // 2, float("inf"))):
        b.q[row, 0, 3] = value
    mass = g.exponential(size=(len(lens), kv, max(lens) + 3)).astype(np.float32)
    scale = dim ** -0.5
    got = ev.accumulate(torch.from_numpy(mass).cuda(), b.q.cuda(), b.cache, *b.device(), max_q=b.max_q, scale=scale,
                        k_exp=b.exps["k_exp"], **kw).cpu().numpy()
    with np.errstate(invalid="ignore"):
        nan = np.isnan(weights(b, mass, scale, **kw)[0])
    # what no such row sees has nothing of it, whatever its values: the same as for any others
    b.q[~b.q.isfinite()] = 1.0
    want, bound = weights(b, mass, scale, **kw)
    assert nan.any() and not nan[:, 1:].any() and (nan[0, 0, :lens[0]].all() == ("causal" in kw))
    assert np.array_equal(np.isnan(got), nan)
    assert (np.abs(got - want) <= bound)[~nan].all()


def test_rows_of_a_pool_and_a_new_output(kvc, ev):
    b = Batch(kvc, [100, 30, 50], [1, 2, 3], 4, 2, 128, 16, 10)
    pool = torch.rand(6, 2, 120, device="cuda")
    at = torch.tensor([4, -1, 0], dtype=torch.int32, device="cuda")
    out = torch.full((6, 3, 130), -5.0, device="cuda")[:, :2, 4:124]
    before = pool.clone()
    kw = dict(max_q=3, k_exp=b.exps["k_exp"])
    got = ev.accumulate(pool, b.q.cuda(), b.cache, *b.device(), rows=at, out=out, **kw)
    assert got is out and torch.equal(pool, before)
    plain = ev.accumulate(pool[[4, 1, 0]], b.q.cuda(), b.cache, *b.device(), **kw)
    assert torch.equal(out[4, :, :100], plain[0, :, :100]) and torch.equal(out[0, :, :50], plain[2, :, :50])
    assert bool((out[4, :, 100:] == -5).all()) and bool((out[[1, 2, 3, 5]] == -5).all())
    for bad in (6, 1 << 30, -(1 << 31)):
        at.fill_(bad)
        ev.accumulate(pool, b.q.cuda(), b.cache, *b.device(), rows=at, **kw)
        assert torch.equal(pool, before)


def test_bad_tables_lengths_and_starts_stay_inside(kvc, ev):
    b = Batch(kvc, [100, 60], [3, 2], 4, 2, 64, 16, 11)
    mass = torch.zeros(2, 2, 200, device="cuda")
    table, lens, starts = b.device()
    for t, n, s in ((torch.full_like(table, 1 << 30), lens, starts), (table, torch.full_like(lens, 1 << 30), starts),
                    (table, -lens, starts), (table, lens, torch.tensor([5, -3, 99], dtype=torch.int32, device="cuda")),
                    (torch.full_like(table, -(1 << 31)), lens, starts)):
        ev.accumulate(mass, b.q.cuda(), b.cache, t, n, s, max_q=3, k_exp=b.exps["k_exp"])
    torch.cuda.synchronize()


def test_long_and_many(kvc, ev):
    # splits of long keys, and rows of many tiles, against the same call cut differently
    b = Batch(kvc, [9000, 4100], [1, 1], 16, 2, 128, 64, 12)
    run_sum = ev.accumulate(torch.zeros(2, 2, 9000, device="cuda"), b.q.cuda(), b.cache, *b.device(), max_q=1,
                            k_exp=b.exps["k_exp"])
    far = ev.accumulate(torch.zeros(2, 2, 9000, device="cuda"), b.q.cuda(), b.cache, *b.device(), max_q=1, max_len=64,
                        k_exp=b.exps["k_exp"])
    assert float((run_sum - far).norm() / far.norm()) < 1e-6
    b = Batch(kvc, [1300], [700], 8, 1, 128, 64, 13)
    whole = ev.accumulate(torch.zeros(1, 1, 1300, device="cuda"), b.q.cuda(), b.cache, *b.device(), max_q=700,
                          k_exp=b.exps["k_exp"])
    parts = torch.zeros(1, 1, 1300, device="cuda")
    table, _, _ = b.device()
    for at in range(0, 700, 100):  # 100 rows at a time, as they would arrive
        i32 = dict(dtype=torch.int32, device="cuda")
        ev.accumulate(parts, b.q[at:at + 100].cuda(), b.cache, table, torch.tensor([700 + at], **i32),
                      torch.tensor([0, 100], **i32), max_q=100, k_exp=b.exps["k_exp"])
    assert float((whole - parts).norm() / whole.norm()) < 1e-6


def chosen(row, n, keep, recent, sinks):
    if n <= keep:
        return list(range(n))
    mid = range(sinks, n - recent)
    key = [np.inf if np.isnan(row[i]) else row[i] for i in mid]
    nan = [np.isnan(row[i]) for i in mid]
    order = sorted(range(len(key)), key=lambda i: (not nan[i], -key[i], i))[:keep - recent - sinks]
    return sorted(list(range(sinks)) + [i + sinks for i in order] + list(range(n - recent, n)))


SELECTS = [  # lens, width, keep, recent, sinks
    ([1], 1, 1, 0, 0), ([10, 3, 0], 12, 4, 1, 1), ([100, 64, 65], 100, 64, 0, 0), ([1000, 999], 1100, 333, 20, 4),
    ([5000, 1024, 1025], 5000, 1024, 256, 64), ([40], 30, 20, 5, 5), ([70], 70, 20, 10, 10), ([70], 70, 20, 20, 0),
    ([9000], 9000, 8999, 0, 0), ([9000], 9000, 1, 0, 0), ([50], 50, 90, 3, 3), ([70000], 70000, 30000, 100, 4),
    ([16385, 20000, 100], 20001, 1500, 30, 2), ([50000], 50000, 49999, 9000, 8500), ([40000, 40000], 40000, 20000, 20000, 0),
    ([33000], 33000, 33000, 5, 5), ([25000, 24000], 25000, 24500, 0, 0),
    ([140000, 20, 16385, 0, 33000, 600], 140000, 700, 30, 2), ([40000, 17, 16384, 300] + 18 * [9], 40000, 16500, 7, 3)]


@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
@pytest.mark.parametrize("lens,width,keep,recent,sinks", SELECTS)
def test_select(ev, lens, width, keep, recent, sinks, kind):
    g = np.random.default_rng(keep)
    mass = g.exponential(size=(len(lens), 3, width)).astype(np.float32) ** 4
    if kind == "ties":  # few different values, and no value at all for most
        mass = np.floor(mass * 2) / 2 * (g.random(mass.shape) < 0.3)
    if kind == "odd":
        mass[g.random(mass.shape) < 0.2] *= -1
        for v in (np.nan, -np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42):
            mass[g.random(mass.shape) < 0.03] = v
    mass = mass.astype(np.float32)
    dev = torch.from_numpy(mass).cuda()
    n32 = torch.tensor(lens, dtype=torch.int32, device="cuda")
    to = torch.full((len(lens), 3, keep + 2), -5.0, device="cuda")
    kept = ev.select(dev, n32, keep, recent=recent, sinks=sinks, mass_out=to).cpu().numpy()
    same = ev.select(dev, n32, keep, recent=recent, sinks=sinks, mass_out=dev)  # in place
    assert np.array_equal(same.cpu().numpy(), kept)
    to, dev = to.cpu().numpy(), dev.cpu().numpy()
    for b, n in enumerate(lens):
        n = min(n, width)
        for h in range(3):
            want = chosen(mass[b, h], n, keep, recent, sinks)
            assert kept[b, h].tolist() == want + [-1] * (keep - len(want))
            m = len(want)
            for t in (to, dev):
                assert np.array_equal(t[b, h, :m], mass[b, h, want], equal_nan=True)
            assert (to[b, h, m:] == -5).all() and np.array_equal(dev[b, h, m:], mass[b, h, m:], equal_nan=True)


def test_select_rows_and_lengths(ev):
    mass = torch.rand(5, 2, 50, device="cuda")
    rows = torch.tensor([3, 9, 0, -2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([40, 40, -7, 40], dtype=torch.int32, device="cuda")
    kept = ev.select(mass, lens, 10, rows=rows)
    assert torch.equal(kept[0], ev.select(mass[3:4], lens[:1], 10)[0])
    assert bool((kept[1:] == -1).all())


@pytest.mark.parametrize("width,keep", [(9000, 300), (40000, 300), (9000, 8800)])
def test_select_of_sequences_with_one_row_in_place(ev, width, keep):
    # each reads sums that others write: any choice, but nothing outside of the outputs
    batch = 40 if width < 10000 else 4
    mass = torch.rand(3, 2, width + 50, device="cuda")
    before = mass.clone()
    kept = torch.full((batch + 2, 2, keep), 7 - (1 << 31), dtype=torch.int32, device="cuda")
    rows = torch.ones(batch, dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), width, dtype=torch.int32, device="cuda")
    ev.select(mass[:, :, :width], lens, keep, recent=5, sinks=3, rows=rows, out=kept[1:-1], mass_out=mass[:, :, :width])
    assert bool((kept[[0, -1]] == 7 - (1 << 31)).all())
    assert torch.equal(mass[[0, 2]], before[[0, 2]]) and torch.equal(mass[1, :, keep:], before[1, :, keep:])


@pytest.mark.parametrize("dim,page,kv", [(64, 16, 3), (128, 64, 2), (256, 32, 1)])
def test_compact(kvc, ev, dim, page, kv):
    lens, keep = [200, 37, 5, 100], 45
    b = Batch(kvc, lens, [1] * 4, kv, kv, dim, page, 14)
    pages = b.cache.k_codes.shape[0]
    more = -(-keep // page)
    cache = kvc.KVCache(*(torch.cat([t, torch.randint(0, 256, (4 * more + 1, *t.shape[1:]), dtype=torch.uint8,
                                                      device="cuda")]) for t in b.cache))
    before = kvc.KVCache(*(t.clone() for t in cache))
    new = torch.arange(pages, pages + 4 * more, dtype=torch.int32).view(4, more).flip(1).contiguous().cuda()
    mass = torch.rand(4, kv, 200, device="cuda")
    table, n32, _ = b.device()
    kept = ev.select(mass, n32, keep, recent=5)
    assert ev.compact(cache, table, kept, new) is cache
    slots_new, slots_old, heads = [], [], []
    for i, n in enumerate(lens):
        for h in range(kv):
            for r, j in enumerate(kept[i, h].tolist()[:min(n, keep)]):
                slots_new.append(int(new[i, r // page]) * page + r % page)
                slots_old.append(int(b.table[i, j // page]) * page + j % page)
                heads.append(h)
    host, old = ({n: t.cpu().numpy() for n, t in c._asdict().items()} for c in (cache, before))
    touched = {n: np.zeros(t.shape, bool) for n, t in host.items()}
    for to, at, h in zip(slots_new, slots_old, heads):
        for part in "kv":
            for x, y in zip(ref.slot_rows(host, part, to), ref.slot_rows(old, part, at)):
                assert np.array_equal(x[h], y[h])
        p, o = to // page, to % page
        touched["k_codes"][p, h, o] = touched["k_scales"][p, h, o] = True
        touched["v_codes"][p, h, o // 16, :, o % 16] = touched["v_scales"][p, h, o // 16, :, o % 16] = True
    for n in host:  # and nothing else
        assert np.array_equal(host[n][~touched[n]], old[n][~touched[n]])


def test_compact_skips_what_is_outside(kvc, ev):
    b = Batch(kvc, [60], [1], 2, 2, 128, 16, 15)
    before = [t.clone() for t in b.cache]
    table, _, _ = b.device()
    i32 = dict(dtype=torch.int32, device="cuda")
    kept = torch.arange(20, **i32).expand(1, 2, 20).contiguous()
    for new in (-1, 1 << 30, b.cache.k_codes.shape[0], -(1 << 31)):
        ev.compact(b.cache, table, kept, torch.full((1, 2), new, **i32))
    for j in (-1, table.shape[1] * 16, (1 << 31) - 1, -(1 << 31)):
        ev.compact(b.cache, table, torch.full_like(kept, j), table)
    ev.compact(b.cache, table, kept, torch.zeros(1, 0, **i32))
    ev.compact(b.cache, table[:, :0].contiguous(), kept, table)
    assert all(torch.equal(x, y) for x, y in zip(b.cache, before))


def test_compact_of_more_sequences_than_a_launch_holds(kvc, ev):
    # 2^24 tiles of 16 tokens: workgroups of 256 threads whose number takes more than 32 bits
    batch, kv, keep, page = 1025, 8, 1 << 15, 1 << 12
    cache = kvc.empty(4, page, kv, 64)
    for t in cache:
        t.copy_(torch.randint(0, 256, t.shape, dtype=torch.uint8, device="cuda"))
    before = [t.clone() for t in cache]
    i32 = dict(dtype=torch.int32, device="cuda")
    kept = torch.full((batch, kv, keep), -1, **i32)
    new = torch.full((batch, keep // page), -1, **i32)
    for b, page_to in ((0, 1), (batch - 2, 2), (batch - 1, 3)):  # the last 16 places of each, from page 0
        kept[b, :, -16:] = torch.arange(b % 7, b % 7 + 16, **i32)
        new[b, -1] = page_to
    ev.compact(cache, torch.zeros(batch, 1, **i32), kept, new)
    for b, page_to in ((0, 1), (batch - 2, 2), (batch - 1, 3)):
        at = slice(b % 7, b % 7 + 16)
        for i in range(2):  # k
            assert torch.equal(cache[i][page_to, :, -16:], before[i][0, :, at])
            assert torch.equal(cache[i][page_to, :, :-16], before[i][page_to, :, :-16])
        old = torch.cat([before[2][0, :, 0], before[2][0, :, 1]], 2)  # v: tiles of 16 tokens
        assert torch.equal(cache[2][page_to, :, -1], old[:, :, at])
        assert torch.equal(cache[2][page_to, :, :-1], before[2][page_to, :, :-1])


def test_attention_after_eviction(kvc, ev):
    """The operators in a row: weights, the choice, the move, and attention over what is left,
    against attention over those tokens' values alone."""
    lens, keep, page, dim, kv, heads = [300, 90], 64, 16, 64, 2, 4
    b = Batch(kvc, lens, [1, 1], heads, kv, dim, page, 16)
    table, n32, starts = b.device()
    q = b.q.cuda()
    mass = torch.zeros(2, kv, 300, device="cuda")
    ev.accumulate(mass, q, b.cache, table, n32, starts, max_q=1, k_exp=b.exps["k_exp"])
    kept = ev.select(mass, n32, keep, recent=8, sinks=2, mass_out=mass)
    cache = kvc.KVCache(*(torch.cat([t, torch.zeros((8, *t.shape[1:]), dtype=torch.uint8, device="cuda")]) for t in b.cache))
    pages = b.cache.k_codes.shape[0]
    new = torch.arange(pages, pages + 8, dtype=torch.int32, device="cuda").view(2, 4)
    ev.compact(cache, table, kept, new)
    left = n32.clamp(max=keep)
    got = kvc.attention(q, cache, new, left, starts, max_q=1, **b.exps)
    host = {n: t.cpu().numpy() for n, t in cache._asdict().items()}
    want, bound = ref.attention(b.q.double().numpy(), host, new.cpu().numpy(), left.tolist(), b.starts, dim ** -0.5,
                                **b.exps)
    assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
    # the next token's weights go onto what was kept
    grown = ev.accumulate(mass, q, cache, new, left, starts, max_q=1, k_exp=b.exps["k_exp"])
    assert bool((grown[:, :, keep - 1] > 0).all())


def test_other_stream_and_graph(kvc, ev):
    b = Batch(kvc, [700, 90], [1, 1], 8, 2, 128, 16, 17)
    args = (b.q.cuda(), b.cache, *b.device())
    kw = dict(max_q=1, max_len=700, k_exp=b.exps["k_exp"])
    work = torch.empty(ev.workspace_bytes(b.cache, total_q=2, heads=8, batch=2, max_q=1, max_len=700), dtype=torch.uint8,
                       device="cuda")
    mass = torch.rand(2, 2, 700, device="cuda")
    out = torch.zeros_like(mass)
    want = ev.accumulate(mass, *args, out=out.clone(), **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ev.accumulate(mass, *args, out=out.clone(), workspace=work, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ev.accumulate(mass, *args, out=out, workspace=work, **kw)
        kept = ev.select(out, args[3], 50, recent=5)
    for i in range(3):
        mass.copy_(torch.rand_like(mass))
        args[0].mul_(-1)
        graph.replay()
        want = ev.accumulate(mass, *args, out=torch.zeros_like(mass), **kw)
        assert torch.equal(out, want) and torch.equal(kept, ev.select(want, args[3], 50, recent=5))


@pytest.mark.parametrize("heads", [8, 32])  # rows of 32 are parted
def test_many_rows_and_long_sums_in_a_graph(kvc, ev, heads):
    # the passes of many rows and the segments of long sums, replayed beside eager calls
    b = Batch(kvc, [400, 90], [70, 90], heads, 2, 128, 16, 19)
    q = b.q.cuda()
    args = (b.cache, *b.device())
    kw = dict(max_q=90, max_len=400, k_exp=b.exps["k_exp"])
    long = torch.rand(2, 2, 30000, device="cuda")
    n32 = torch.tensor([30000, 17000], dtype=torch.int32, device="cuda")
    work = torch.empty(ev.workspace_bytes(b.cache, total_q=160, heads=heads, batch=2, max_q=90, max_len=400), dtype=torch.uint8,
                       device="cuda")
    space = torch.empty(ev.select_workspace_bytes(long, 2, 5000), dtype=torch.uint8, device="cuda")
    out = torch.zeros(2, 2, 400, device="cuda")
    kept = ev.select(long, n32, 5000, recent=64, workspace=space)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ev.accumulate(out, q, *args, workspace=work, **kw)
        ev.select(long, n32, 5000, recent=64, out=kept, workspace=space)
    for i in range(3):
        q.mul_(1.1)
        long.copy_(long.roll(1000, 2))
        out.zero_()
        graph.replay()
        want = ev.accumulate(torch.zeros_like(out), q, *args, **kw)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(kept, ev.select(long, n32, 5000, recent=64))


def test_padded_batches(kvc, ev):
    # rows of q before the first sequence and behind the last, and sequences without rows
    b = Batch(kvc, [80, 50, 33], [5, 0, 40], 4, 2, 64, 16, 20)
    table, lens, _ = b.device()
    q = torch.randn(60, 4, 64, device="cuda").bfloat16()
    starts = torch.tensor([7, 12, 12, 52], dtype=torch.int32, device="cuda")
    mass = torch.rand(3, 2, 100, device="cuda")
    got = ev.accumulate(mass.clone(), q, b.cache, table, lens, starts, max_q=40, k_exp=b.exps["k_exp"])
    close = torch.cat([q[7:12], q[12:52]])
    want = ev.accumulate(mass.clone(), close, b.cache, table, lens,
                         torch.tensor([0, 5, 5, 45], dtype=torch.int32, device="cuda"), max_q=40, k_exp=b.exps["k_exp"])
    assert torch.equal(got, want) and torch.equal(got[1], mass[1])


def test_refusals(kvc, ev):
    b = Batch(kvc, [40, 20], [1, 1], 4, 2, 64, 16, 18)
    mass = torch.zeros(2, 2, 40, device="cuda")
    table, lens, starts = b.device()
    ok = dict(mass=mass, q=b.q.cuda(), cache=b.cache, page_table=table, seq_lens=lens, q_starts=starts, max_q=1)
    for kw in (dict(mass=mass.double()), dict(mass=mass[:1]), dict(mass=mass[:, :1]), dict(mass=mass.cpu()),
               dict(mass=mass[:, :, ::2]), dict(out=mass[:, :, :39]), dict(q=b.q), dict(q=ok["q"][:, :3]), dict(window=-1),
               dict(causal=False, window=3), dict(scale=-1.0), dict(scale=float("nan")), dict(seq_lens=lens.long()),
               dict(rows=lens.long()), dict(rows=lens[:1]), dict(k_exp=65), dict(max_q=-1), dict(max_len=-1),
               dict(out=mass[:1].expand(2, 2, 40)), dict(mass=mass[:1].expand(2, 2, 40)), dict(workspace=torch.zeros(1, dtype=torch.uint8, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            ev.accumulate(**{**ok, **kw})
    wide = torch.zeros(1, 2, 40000, device="cuda")
    assert ev.select_workspace_bytes(wide, 1, 10) > 0 and ev.select_workspace_bytes(mass, 2, 10) == 0
    with pytest.raises(ValueError, match="workspace"):
        ev.select(wide, lens[:1], 10, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    for kw in (dict(keep=-1), dict(keep=3, recent=4), dict(keep=5, recent=3, sinks=3), dict(sinks=-1), dict(recent=-1),
               dict(seq_lens=lens.long()), dict(mass_out=mass[:, :, :3]), dict(mass_out=mass[:1].expand(2, 2, 40)), dict(out=torch.zeros(2, 2, 3, device="cuda")),
               dict(mass=mass.cpu())):
        with pytest.raises((ValueError, RuntimeError)):
            ev.select(**{**dict(mass=mass, seq_lens=lens, keep=10), **kw})
    kept = ev.select(mass, lens, 10)
    for args in ((table[:1], kept, table), (table, kept[:, :1].contiguous(), table), (table, kept.long(), table),
                 (table, kept, table.long()), (table.cpu(), kept, table), (table, kept, table[0])):
        with pytest.raises(ValueError):
            ev.compact(b.cache, *args)


def test_sums_whose_rows_meet_are_refused(kvc, ev):
    # strides that are wide enough each, and rows of two sequences in one place
    b = Batch(kvc, [40, 20], [1, 1], 4, 2, 64, 16, 18)
    args = (b.q.cuda(), b.cache, *b.device())
    kw = dict(max_q=1, k_exp=b.exps["k_exp"])
    buffer, mass = torch.zeros(200, device="cuda"), torch.zeros(2, 2, 40, device="cuda")
    bad, good = (buffer.as_strided((2, 2, 40), (s, 40, 1)) for s in (40, 80))
    for call in (lambda t: ev.accumulate(mass, *args, out=t, **kw), lambda t: ev.accumulate(t, *args, **kw),
                 lambda t: ev.select(mass, args[3], 10, mass_out=t)):
        with pytest.raises(ValueError, match="overlap"):
            call(bad)
        call(good)
    # heads before sequences
    turned = torch.zeros(2, 2, 40, device="cuda").transpose(0, 1)
    assert torch.equal(ev.accumulate(mass, *args, out=turned, **kw), ev.accumulate(mass.clone(), *args, **kw))
