"""The eviction entry points' C ABI: exports of include/if4_kv_evict.h, and refusals, which
come before any HIP call (so these run without a GPU)."""
import math
import os
import random
import re

import pytest

from test_kv_abi import BAD_ARGS, BAD_BUFFERS, BAD_CACHES, args, cache

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "if4_kv_evict.h")
LIB = os.path.join(ROOT, "adaptive_block_scaled_amd", "libif4.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libif4.so not built")

OK, NULL, SHAPE, ALIGN, DTYPE, RANGE = range(6)
FAKE = 0x100000  # 16-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def kvc():
    from adaptive_block_scaled_amd import kv_cache
    return kv_cache


@pytest.fixture(scope="module")
def ev():
    from adaptive_block_scaled_amd import kv_evict
    return kv_evict


def mass(ev, **kw):
    base = dict(in_=FAKE, in_stride_row=80, in_stride_head=40, out=FAKE, out_stride_row=80, out_stride_head=40,
                rows=None, mass_rows=2, width=40)
    base.update(kw)
    return ev._Mass(**base)


BAD_MASS = [(dict(mass_rows=-1), SHAPE), (dict(mass_rows=1), SHAPE), (dict(width=-1), SHAPE), (dict(width=1 << 31), SHAPE),
            (dict(mass_rows=1 << 31), SHAPE), (dict(in_=None), NULL), (dict(in_=FAKE + 2), ALIGN), (dict(out=FAKE + 1), ALIGN),
            (dict(rows=FAKE + 2), ALIGN)]


def test_exports_every_declared_symbol(ev):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(if4_\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(ev.EXPORTS)
    for n in names:
        assert hasattr(ev.lib, n), n


def test_weights_refusals(kvc, ev):
    def call(a=None, c=None, m=None, ws=FAKE, size=1 << 40):
        return ev.lib.if4_kv_weights(cache(kvc) if c is None else c, args(kvc) if a is None else a,
                                     mass(ev) if m is None else m, ws, size, None)
    for kw, st in BAD_CACHES + BAD_BUFFERS:
        assert call(c=cache(kvc, **kw)) == st, kw
    for kw, st in BAD_ARGS:
        assert call(args(kvc, **kw)) == st, kw
        assert ev.lib.if4_kv_weights_workspace(cache(kvc), args(kvc, **kw)) == -st
        assert ev.lib.if4_kv_weights_workspace_most(cache(kvc), args(kvc, **kw)) == -st
    for kw, st in BAD_MASS + [(dict(out=None), NULL)]:
        assert call(m=mass(ev, **kw)) == st, kw
    f = ev.lib.if4_kv_weights
    assert f(None, args(kvc), mass(ev), FAKE, 1 << 40, None) == NULL
    assert f(cache(kvc), None, mass(ev), FAKE, 1 << 40, None) == NULL
    assert f(cache(kvc), args(kvc), None, FAKE, 1 << 40, None) == NULL
    for n in ("q", "page_table", "seq_lens", "q_starts"):
        assert call(args(kvc, **{n: None})) == NULL, n
        assert call(args(kvc, **{n: FAKE + 2})) == ALIGN, n
    for n in ("q_stride_token", "q_stride_head"):
        assert call(args(kvc, **{n: 132})) == ALIGN, n
    need = ev.lib.if4_kv_weights_workspace(cache(kvc), args(kvc))
    assert need > 0
    assert call(ws=None) == NULL and call(size=need - 1) == SHAPE and call(ws=FAKE + 8) == ALIGN
    # nothing to compute, or nowhere to put it
    for kw in (dict(batch=0), dict(total_q=0), dict(max_q=0)):
        assert call(args(kvc, q=None, **kw), ws=None) == OK
    assert call(c=cache(kvc, pages=0, k_codes=None)) == OK
    assert call(m=mass(ev, width=0, in_=None)) == OK and call(m=mass(ev, rows=FAKE, mass_rows=0, in_=None)) == OK


def test_select_refusals(ev):
    def call(m=None, lens=FAKE, batch=2, kv=2, keep=10, recent=2, sinks=1, kept=FAKE, ws=None, size=0):
        return ev.lib.if4_kv_select(mass(ev) if m is None else m, lens, batch, kv, keep, recent, sinks, kept, ws, size, None)
    for kw, st in BAD_MASS:
        assert call(mass(ev, **kw)) == st, kw
    for kw in (dict(batch=-1), dict(kv=0), dict(kv=1 << 17), dict(batch=1 << 31), dict(keep=-1), dict(keep=1 << 31)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(recent=-1), dict(sinks=-1), dict(recent=11), dict(sinks=9), dict(recent=1 << 62, sinks=1 << 62)):
        assert call(**kw) == RANGE, kw
    assert call(lens=None) == NULL and call(kept=None) == NULL
    assert call(lens=FAKE + 2) == ALIGN and call(kept=FAKE + 1) == ALIGN
    assert ev.lib.if4_kv_select(None, FAKE, 2, 2, 10, 0, 0, FAKE, None, 0, None) == NULL
    f = ev.lib.if4_kv_select_workspace
    for kw in (dict(batch=-1), dict(kv_heads=0), dict(keep=-1), dict(keep=1 << 31)):
        assert f(mass(ev), *{**dict(batch=2, kv_heads=2, keep=10), **kw}.values()) == -SHAPE
    assert f(None, 2, 2, 10) == -NULL and f(mass(ev, width=-1), 2, 2, 10) == -SHAPE and f(mass(ev), 2, 2, 10) == 0
    wide = dict(width=100000, in_stride_row=200000, in_stride_head=100000, out_stride_row=200000, out_stride_head=100000)
    need = f(mass(ev, **wide), 2, 2, 10)
    assert 0 < need <= 8 << 20
    assert call(mass(ev, **wide), size=need) == NULL and call(mass(ev, **wide), ws=FAKE, size=need - 1) == SHAPE
    assert call(mass(ev, **wide), ws=FAKE + 8, size=need) == ALIGN
    assert call(batch=0, lens=None) == OK and call(keep=0, recent=0, sinks=0, kept=None) == OK


def test_compact_refusals(kvc, ev):
    def call(c=None, table=FAKE, ts=3, kept=FAKE, batch=2, keep=20, new=FAKE, ns=2):
        return ev.lib.if4_kv_compact(cache(kvc) if c is None else c, table, ts, kept, batch, keep, new, ns, None)
    for kw, st in BAD_CACHES + BAD_BUFFERS:
        assert call(cache(kvc, **kw)) == st, kw
    for kw in (dict(batch=-1), dict(keep=-1), dict(ts=-1), dict(ns=-1), dict(keep=1 << 31), dict(ts=1 << 31), dict(ns=1 << 31),
               dict(batch=1 << 31), dict(batch=1 << 20, keep=1 << 20)):
        assert call(**kw) == SHAPE, kw
    for n in ("table", "kept", "new"):
        assert call(**{n: None}) == NULL and call(**{n: FAKE + 2}) == ALIGN, n
    assert ev.lib.if4_kv_compact(None, FAKE, 3, FAKE, 2, 20, FAKE, 2, None) == NULL
    for kw in (dict(batch=0), dict(keep=0), dict(ts=0), dict(ns=0)):
        assert call(table=None, **kw) == OK


def test_one_workspace_is_enough_for_all_smaller_calls(kvc, ev):
    need, most = ev.lib.if4_kv_weights_workspace, ev.lib.if4_kv_weights_workspace_most
    rng = random.Random(7)

    def log(hi):
        return min(hi, max(1, round(math.exp(rng.uniform(0, math.log(hi + 1))))))
    for _ in range(1000):
        kv = rng.choice([1, 2, 3, 8])
        heads, dim = kv * rng.choice([1, 2, 4, 7, 8, 40]), rng.choice([64, 128, 256])
        c = kvc._Cache(pages=1000, page_size=64, kv_heads=kv, head_dim=dim)
        top = dict(batch=log(600), total_q=log(20000), max_q=log(9000), max_len=log(1 << 20))

        def size(f, **kw):
            return f(c, kvc._Attention(heads=heads, scale=1.0, causal=1, **kw))
        bound = size(most, **top)
        for name in top:
            assert size(most, **{**top, name: 2 * top[name]}) >= bound
        for _ in range(20):
            call = {n: rng.choice([log(v), v]) for n, v in top.items()}
            assert 0 < size(need, **call) <= bound


def test_binding_needs_gpu_tensors(kvc, ev):
    import torch
    c = kvc.empty(2, 16, 2, 64, device="cpu")
    m, i = torch.zeros(1, 2, 32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ev.accumulate(m, torch.zeros(1, 2, 64).bfloat16(), c, i[None], i, i, max_q=1)
    with pytest.raises(ValueError, match="CUDA"):
        ev.select(m, i, 4)
    with pytest.raises(ValueError, match="CUDA"):
        ev.compact(c, i[None], i[None, None], i[None])


def test_rows_of_sums_that_overlap(ev):
    # [2 sequences, 3 heads, 40]: wide enough strides of each may still meet one another's rows
    import torch
    buffer = torch.zeros(1000)
    mass = torch.zeros(2, 3, 40)
    for strides in ((40, 40), (80, 40), (100, 40), (40, 60), (39, 200), (200, 39), (0, 40), (120, 0)):
        with pytest.raises(ValueError, match="overlap"):
            ev._mass(mass, buffer.as_strided((2, 3, 40), (*strides, 1)), None, 2, torch.device("cpu"))
    for strides in ((120, 40), (40, 80), (150, 45), (50, 100)):
        m = ev._mass(mass, buffer.as_strided((2, 3, 40), (*strides, 1)), None, 2, torch.device("cpu"))
        assert (m.out_stride_row, m.out_stride_head) == strides
    for shape in ((1, 3, 40), (2, 1, 40)):  # what nothing is apart by has any stride
        ev._mass(mass[:shape[0], :shape[1]], buffer.as_strided(shape, (40, 40, 1)), None, shape[0], torch.device("cpu"))
