"""The C ABI of the norm and rotation of q and k: exports of include/if4_qk.h, and refusals,
which come before any HIP call (so these run without a GPU)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "if4_qk.h")
LIB = os.path.join(ROOT, "adaptive_block_scaled_amd", "libif4.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libif4.so not built")

OK, NULL, SHAPE, ALIGN, DTYPE, RANGE = range(6)
FAKE = 0x100000  # 16-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def qk():
    from adaptive_block_scaled_amd import qk
    return qk


def test_exports_every_declared_symbol(qk):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(if4_\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(qk.EXPORTS)
    for n in names:
        assert hasattr(qk.lib, n), n


def args(qk, part="q", **kw):
    a = qk._Args(table=FAKE, positions=FAKE, tokens=3, head_dim=64, rotary=64, table_rows=10, eps=1e-6,
                 interleaved=0, dtype=0, out_dtype=1)
    for p, heads in ((a.q, 4), (a.k, 2)):
        p.x = p.g = p.y = p.weight = p.d_weight = FAKE
        p.x_stride_token = p.g_stride_token = p.y_stride_token = 512
        p.x_stride_head = p.g_stride_head = p.y_stride_head = 64
        p.heads = heads
    for name, v in kw.items():
        setattr(getattr(a, part) if hasattr(a.q, name) else a, name, v)
    return a


SIZES = [(dict(head_dim=0), SHAPE), (dict(head_dim=60), SHAPE), (dict(head_dim=264), SHAPE), (dict(rotary=-8), SHAPE),
         (dict(rotary=72), SHAPE), (dict(rotary=12), SHAPE), (dict(rotary=24), SHAPE), (dict(rotary=20, interleaved=1), SHAPE), (dict(tokens=-1), SHAPE), (dict(tokens=1 << 32), SHAPE),
         (dict(table_rows=-1), SHAPE), (dict(heads=-1), SHAPE), (dict(heads=1 << 17), SHAPE), (dict(eps=-1.0), RANGE),
         (dict(eps=float("inf")), RANGE), (dict(eps=float("nan")), RANGE), (dict(dtype=2), DTYPE),
         (dict(out_dtype=-1), DTYPE), (dict(interleaved=2), DTYPE)]


@pytest.mark.parametrize("part", ["q", "k"])
def test_refusals(qk, part):
    need = qk.lib.if4_norm_rotate_backward_workspace(args(qk))
    assert 0 < need <= 8 << 20

    def calls(**kw):
        a = args(qk, part, **kw)
        return (qk.lib.if4_norm_rotate(a, None), qk.lib.if4_norm_rotate_backward(a, FAKE, need, None))
    for kw, st in SIZES:
        assert calls(**kw) == (st, st), kw
        assert qk.lib.if4_norm_rotate_backward_workspace(args(qk, part, **kw)) == -st
    for name in ("x", "y", "weight", "table", "positions"):
        assert calls(**{name: None}) == (NULL, NULL), name
        assert calls(**{name: FAKE + 4}) == (ALIGN, ALIGN), name
    for name in ("x_stride_token", "x_stride_head", "y_stride_token", "y_stride_head"):
        assert calls(**{name: 65}) == (ALIGN, ALIGN), name
    back = dict(workspace=FAKE, size=need)
    for kw, st in ((dict(g=None), NULL), (dict(g=FAKE + 8), ALIGN), (dict(d_weight=None), NULL), (dict(d_weight=FAKE + 2), ALIGN),
                   (dict(g_stride_token=60), ALIGN), (dict(g_stride_head=4), ALIGN)):
        assert qk.lib.if4_norm_rotate_backward(args(qk, part, **kw), *back.values(), None) == st, kw
    f = qk.lib.if4_norm_rotate_backward
    assert f(args(qk), None, need, None) == NULL and f(args(qk), FAKE, need - 1, None) == SHAPE
    assert f(args(qk), FAKE + 8, need, None) == ALIGN
    assert f(None, FAKE, need, None) == NULL and qk.lib.if4_norm_rotate(None, None) == NULL
    assert qk.lib.if4_norm_rotate_backward_workspace(None) == -NULL
    # nothing to do
    assert qk.lib.if4_norm_rotate(args(qk, tokens=0, positions=None), None) == OK
    a = args(qk)
    a.q.heads = a.k.heads = 0
    assert qk.lib.if4_norm_rotate(a, None) == OK and f(a, None, 0, None) == OK


def test_binding_needs_gpu_tensors(qk):
    import torch
    x, w, pos = torch.zeros(3, 2, 64), torch.ones(64), torch.zeros(3, dtype=torch.int64)
    table = qk.rotation_table(5, 64, device="cpu")
    assert table.shape == (5, 64) and bool((table[0, :32] == 1).all()) and not bool(table[0, 32:].any())
    with pytest.raises(ValueError, match="CUDA"):
        qk.norm_rotate(x, x, w, w, table, pos)
    with pytest.raises(ValueError, match="CUDA"):
        qk.norm_rotate_backward(x, x, x, x, w, w, table, pos)
