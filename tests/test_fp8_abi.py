"""The FP8 entry points' C ABI: exports of include/if4_fp8.h, and refusals, which come
before any HIP call (so these run without a GPU); and the oracle's own pins."""
import os
import re

import numpy as np
import pytest

import fp8_reference as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "if4_fp8.h")
LIB = os.path.join(ROOT, "adaptive_block_scaled_amd", "libif4.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libif4.so not built")

OK, NULL, SHAPE, ALIGN, DTYPE, RANGE = range(6)
FAKE = 0x100000  # 16-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def fp8():
    from adaptive_block_scaled_amd import fp8
    return fp8


def test_exports_every_declared_symbol(fp8):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = re.findall(r"^\s*(?:int|int64_t)\s+(if4_\w+)\s*\(", text, flags=re.M)
    assert sorted(names) == sorted(fp8.EXPORTS)
    for n in names:
        assert hasattr(fp8.lib, n), n


@pytest.mark.parametrize("name", ["if4_fp8_quantize", "if4_fp8_quantize_t"])
def test_quantize_refusals(fp8, name):
    def call(x=FAKE, dt=1, rows=32, cols=64, ld=64, square=0, codes=FAKE, scales=FAKE):
        return getattr(fp8.lib, name)(x, dt, rows, cols, ld, square, codes, scales, None)
    assert call(dt=2) == DTYPE and call(square=2) == DTYPE and call(square=-1) == DTYPE
    assert call(rows=-16) == SHAPE and call(cols=-16) == SHAPE and call(ld=63) == SHAPE
    along = dict(cols=72, ld=72) if name == "if4_fp8_quantize" else dict(rows=40)
    assert call(**along) == SHAPE
    assert call(rows=1 << 32) == SHAPE and call(cols=1 << 32, ld=1 << 32) == SHAPE and call(ld=1 << 41) == SHAPE
    assert call(rows=1 << 31, cols=1 << 10, ld=1 << 10) == SHAPE  # more blocks than a grid has
    assert call(x=None) == NULL and call(codes=None) == NULL and call(scales=None) == NULL
    assert call(x=FAKE + 8) == ALIGN and call(codes=FAKE + 8) == ALIGN
    assert call(ld=68) == ALIGN and call(dt=0, ld=66) == ALIGN
    assert call(rows=0, x=None) == OK and call(cols=0, x=None) == OK


def test_gemm_refusals(fp8):
    def call(m=8, n=24, k=48, ac=FAKE, asc=FAKE, wc=FAKE, ws=FAKE, square=0, c=FAKE, dt=1, ld=24, work=FAKE, size=1 << 40):
        return fp8.lib.if4_fp8_gemm(ac, asc, wc, ws, square, m, n, k, c, dt, ld, work, size, None)
    assert call(dt=2) == DTYPE and call(square=3) == DTYPE
    for kw in (dict(m=-1), dict(n=-1), dict(k=-16), dict(k=40), dict(ld=23), dict(m=1 << 32), dict(n=1 << 32, ld=1 << 33),
               dict(k=1 << 23), dict(ld=1 << 41)):
        assert call(**kw) == SHAPE, kw
    for name in ("ac", "asc", "wc", "ws", "c"):
        assert call(**{name: None}) == NULL
    for name in ("ac", "wc"):
        assert call(**{name: FAKE + 8}) == ALIGN
    assert call(c=FAKE + 1) == ALIGN and call(c=FAKE + 2, dt=0) == ALIGN
    assert call(m=0, c=None) == OK and call(n=0, c=None) == OK


def test_workspace(fp8):
    f = fp8.lib.if4_fp8_gemm_workspace
    for bad in ((-1, 1, 16), (1, -1, 16), (1, 1, -16), (1, 1, 24), (1 << 32, 1, 16), (1, 1, 1 << 23)):
        assert f(*bad) == -SHAPE, bad
    for nothing in ((0, 8, 16), (8, 0, 16), (8, 8, 0)):
        assert f(*nothing) == 0
    # whatever is asked for: a call without it, or with less, is refused
    for m, n, k in ((1, 6144, 4096), (64, 4096, 4096), (16, 100, 8192), (1021, 5003, 4112), (100, 100, 28672), (300, 300, 65536)):
        need = f(m, n, k)
        assert 0 <= need <= 256 << 20
        if need:
            args = (FAKE, FAKE, FAKE, FAKE, 1, m, n, k, FAKE, 1, n)
            assert fp8.lib.if4_fp8_gemm(*args, None, need, None) == NULL
            assert fp8.lib.if4_fp8_gemm(*args, FAKE, need - 1, None) == SHAPE
            assert fp8.lib.if4_fp8_gemm(*args, FAKE + 8, need, None) == ALIGN
    assert f(1 << 31, 1 << 31, 1 << 22) == 0 and f(1 << 31, 1, 1 << 22) >= 0  # the largest sizes


def test_binding_needs_gpu_tensors(fp8):
    import torch
    x, u8 = torch.zeros(16, 32), torch.zeros(16, 32, dtype=torch.uint8)
    for f in (fp8.quantize, fp8.quantize_t):
        with pytest.raises(ValueError, match="CUDA"):
            f(x)
    with pytest.raises(ValueError, match="CUDA"):
        fp8.gemm(u8, u8[:, :1], u8, u8[:, :1])


def test_the_oracle_on_worked_blocks():
    # 448 is the largest code (0x7E) at exponent 0; 449 is 224.5 at exponent 1, next to 224
    # (0x76); half of the smallest code, and one and a half of it, are ties that go to even
    x = np.zeros((4, 128))
    x[0, :3] = 448, -448, 2.0 ** -10
    x[1, :3] = 449, 3 * 2.0 ** -9, -0.0
    x[2, 5] = np.inf
    codes, scales = ref.quantize(x)
    assert scales[:, 0].tolist() == [127, 128, 255, 0]
    assert codes[0, :4].tolist() == [0x7E, 0xFE, 0, 0]
    assert codes[1, :4].tolist() == [0x76, 2, 0x80, 0]
    assert (codes[2] == 0x7F).all() and not codes[3].any()
    v = ref.values(codes, scales)
    assert v[0, 0] == 448 and v[1, 0] == 448 and v[1, 1] == 2.0 ** -7 and np.isnan(v[2]).all()
    # the same values from a square and from its transpose
    g = np.random.default_rng(1).standard_normal((200, 144))
    a, b = ref.quantize(g, True), ref.quantize(g.T, True)
    assert (a[0].T == b[0]).all() and (a[1].T == b[1]).all()
