"""The KV cache's C ABI: exports of include/if4_kv.h, and its refusals, which
come before any HIP call (so these run without a GPU).  The Python binding
refuses tensors that are not on a GPU."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "if4_kv.h")
LIB = os.path.join(ROOT, "adaptive_block_scaled_amd", "libif4.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libif4.so not built")

OK, NULL, SHAPE, ALIGN, DTYPE, RANGE = range(6)
FAKE = 0x100000  # 16-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def kvc():
    from adaptive_block_scaled_amd import kv_cache
    return kv_cache


def test_exports_every_declared_symbol(kvc):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(if4_\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(kvc.EXPORTS)
    for n in names:
        assert hasattr(kvc.lib, n), n


def cache(kvc, **kw):
    base = dict(k_codes=FAKE, k_scales=FAKE, v_codes=FAKE, v_scales=FAKE, pages=4, page_size=16,
                kv_heads=2, head_dim=128, k_exp=0, v_exp=0)
    base.update(kw)
    return kvc._Cache(**base)


BAD_CACHES = [(dict(head_dim=96), SHAPE), (dict(head_dim=0), SHAPE), (dict(page_size=24), SHAPE),
              (dict(page_size=0), SHAPE), (dict(page_size=-16), SHAPE), (dict(pages=-1), SHAPE),
              (dict(kv_heads=0), SHAPE), (dict(kv_heads=65536), SHAPE), (dict(pages=1 << 31), SHAPE),
              (dict(k_exp=65), RANGE), (dict(v_exp=-65), RANGE)]
BAD_BUFFERS = [(dict(k_codes=None), NULL), (dict(v_scales=None), NULL), (dict(v_codes=FAKE + 8), ALIGN),
               (dict(k_scales=FAKE + 4), ALIGN)]


def test_append_refusals(kvc):
    def call(c=None, k=FAKE, v=FAKE, dt=1, n=3, st=(256, 128, 256, 128), slots=FAKE, mode=0):
        return kvc.lib.if4_kv_append(cache(kvc) if c is None else c, k, v, dt, n, *st, slots, mode, None)
    for kw, st in BAD_CACHES + BAD_BUFFERS:
        assert call(cache(kvc, **kw)) == st, kw
    assert kvc.lib.if4_kv_append(None, FAKE, FAKE, 1, 3, 8, 8, 8, 8, FAKE, 0, None) == NULL
    assert call(dt=2) == DTYPE and call(mode=3) == DTYPE and call(mode=-1) == DTYPE
    assert call(n=-1) == SHAPE
    assert call(k=None) == NULL and call(v=None) == NULL and call(slots=None) == NULL
    assert call(k=FAKE + 8) == ALIGN and call(v=FAKE + 2) == ALIGN and call(slots=FAKE + 4) == ALIGN
    for i in range(4):
        st = [256, 128, 256, 128]
        st[i] += 4
        assert call(st=st) == ALIGN           # 8 bytes in bf16
        assert call(st=[s + 2 for s in st], dt=0) == ALIGN
    # nothing to write
    assert call(n=0, k=None) == OK
    assert call(cache(kvc, pages=0, k_codes=None)) == OK


def test_read_refusals(kvc):
    def call(c=None, slots=FAKE, n=3, k=FAKE, v=FAKE, dt=1):
        return kvc.lib.if4_kv_read(cache(kvc) if c is None else c, slots, n, k, v, dt, None)
    for kw, st in BAD_CACHES + BAD_BUFFERS:
        assert call(cache(kvc, **kw)) == st, kw
    assert kvc.lib.if4_kv_read(None, FAKE, 1, FAKE, FAKE, 1, None) == NULL
    assert call(dt=7) == DTYPE and call(n=-2) == SHAPE
    assert call(k=None) == NULL and call(v=None) == NULL and call(slots=None) == NULL
    assert call(k=FAKE + 4) == ALIGN and call(v=FAKE + 8) == ALIGN and call(slots=FAKE + 1) == ALIGN
    assert call(n=0, k=None) == OK


def args(kvc, **kw):
    base = dict(q=FAKE, out=FAKE, q_stride_token=512, q_stride_head=128, out_stride_token=512,
                out_stride_head=128, page_table=FAKE, table_stride=3, seq_lens=FAKE, q_starts=FAKE,
                batch=2, total_q=5, heads=4, max_q=3, max_len=40, window=0, sinks=0, scale=0.1, causal=1)
    base.update(kw)
    return kvc._Attention(**base)


BAD_ARGS = [(dict(batch=-1), SHAPE), (dict(total_q=-1), SHAPE), (dict(max_q=-1), SHAPE),
            (dict(max_len=-1), SHAPE), (dict(table_stride=-1), SHAPE), (dict(heads=0), SHAPE),
            (dict(heads=3), SHAPE), (dict(total_q=1 << 30), SHAPE), (dict(batch=1 << 30), SHAPE),
            (dict(window=-1), RANGE), (dict(sinks=-1), RANGE), (dict(causal=0, window=5), RANGE),
            (dict(causal=0, sinks=5), RANGE), (dict(scale=float("nan")), RANGE),
            (dict(scale=float("inf")), RANGE), (dict(scale=-0.5), RANGE)]


def test_attention_refusals(kvc):
    def call(a=None, c=None, ws=FAKE, size=1 << 40):
        return kvc.lib.if4_kv_attention(cache(kvc) if c is None else c, args(kvc) if a is None else a,
                                        ws, size, None)
    for kw, st in BAD_CACHES + BAD_BUFFERS:
        assert call(c=cache(kvc, **kw)) == st, kw
    for kw, st in BAD_ARGS:
        assert call(args(kvc, **kw)) == st, kw
    assert kvc.lib.if4_kv_attention(None, args(kvc), None, 0, None) == NULL
    assert kvc.lib.if4_kv_attention(cache(kvc), None, None, 0, None) == NULL
    for n in ("q", "out", "page_table", "seq_lens", "q_starts"):
        assert call(args(kvc, **{n: None})) == NULL, n
        assert call(args(kvc, **{n: FAKE + 2})) == ALIGN, n
    for n in ("q_stride_token", "q_stride_head", "out_stride_token", "out_stride_head"):
        assert call(args(kvc, **{n: 132})) == ALIGN, n
    long = dict(batch=1, total_q=1, max_q=1, max_len=100000)
    need = kvc.lib.if4_kv_attention_workspace(cache(kvc), args(kvc, **long))
    assert need > 0
    assert call(args(kvc, **long), ws=None) == NULL
    assert call(args(kvc, **long), size=need - 1) == SHAPE
    assert call(args(kvc, **long), ws=FAKE + 8) == ALIGN
    # nothing to compute
    for kw in (dict(batch=0), dict(total_q=0), dict(max_q=0)):
        assert call(args(kvc, q=None, **kw)) == OK


def test_workspace_refusals(kvc):
    f = kvc.lib.if4_kv_attention_workspace
    for kw, st in BAD_CACHES:
        assert f(cache(kvc, **kw), args(kvc)) == -st, kw
    for kw, st in BAD_ARGS:
        assert f(cache(kvc), args(kvc, **kw)) == -st, kw
    assert f(None, args(kvc)) == -NULL and f(cache(kvc), None) == -NULL
    assert f(cache(kvc), args(kvc, batch=0)) == 0
    # no more rows than there are: the hint does not grow the workspace
    assert f(cache(kvc), args(kvc, max_q=1 << 40)) == f(cache(kvc), args(kvc, max_q=5))


def test_binding_needs_gpu_tensors(kvc):
    import torch
    c = kvc.empty(2, 16, 2, 64, device="cpu")
    assert [tuple(t.shape) for t in c] == [(2, 2, 16, 32), (2, 2, 16, 4), (2, 2, 1, 16, 16, 2), (2, 2, 1, 4, 16)]
    x, slots = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.append(c, x, x, slots)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.read(c, slots)
    with pytest.raises(ValueError, match="CUDA"):
        kvc.attention(x, c, slots, slots, slots, max_q=1)
    for kw in (dict(head_dim=80), dict(page_size=8), dict(page_size=0)):
        with pytest.raises(ValueError, match=next(iter(kw))):
            kvc.empty(**{**dict(pages=1, page_size=16, kv_heads=1, head_dim=64, device="cpu"), **kw})
