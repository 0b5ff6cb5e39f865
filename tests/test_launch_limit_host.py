"""Calls of more work than one launch holds: HIP counts the threads of a grid in 32 bits and
drops what lies above without an error, so every entry point refuses them before it
launches anything (these run without a GPU; no address is dereferenced)."""
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "adaptive_block_scaled_amd", "libif4.so")

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libif4.so not built")

SHAPE = 2
FAKE = 0x100000
BF16, F32 = 1, 0
WIDE = 1 << 36  # groups of 16: more than 2^32 threads of any kernel


@pytest.fixture(scope="module")
def lib():
    from adaptive_block_scaled_amd import decoder_attention  # declares all entry points
    from adaptive_block_scaled_amd.if4 import lib
    return lib


def test_quantize_and_dequantize(lib):
    for dt in (BF16, F32):
        if dt == BF16:  # (fp32 rows are gone through in a loop)
            assert lib.if4_quantize_mode(FAKE, dt, WIDE, 16, 16, FAKE, FAKE, 0, 0, None) == SHAPE
            assert lib.if4_quantize_rht(FAKE, dt, WIDE, 16, 16, 1, FAKE, FAKE, 0, 0, None) == SHAPE
        assert lib.if4_quantize_t(FAKE, dt, 16, WIDE, WIDE, FAKE, FAKE, 0, 0, None) == SHAPE
        assert lib.if4_quantize_t(FAKE, dt, WIDE, 8, 8, FAKE, FAKE, 0, 0, None) == SHAPE
        assert lib.if4_dequantize(FAKE, FAKE, WIDE, 16, 0, FAKE, dt, 16, None) == SHAPE
        for bits in (3, 6):
            assert lib.if4_quantize_ifn(bits, FAKE, dt, WIDE, 16, 16, FAKE, FAKE, 0, 0, None) == SHAPE
            assert lib.if4_dequantize_ifn(bits, FAKE, FAKE, WIDE, 16, 0, FAKE, dt, 16, None) == SHAPE
    assert lib.if4_gemm(FAKE, FAKE, 0, FAKE, FAKE, 0, 1 << 31, 1 << 31, 16, FAKE, 1 << 31, None) == SHAPE


def test_fp8(lib):
    for dt in (BF16, F32):
        assert lib.if4_fp8_quantize(FAKE, dt, 1 << 29, 16, 16, 0, FAKE, FAKE, None) == SHAPE
        assert lib.if4_fp8_quantize(FAKE, dt, 1 << 31, 16, 16, 1, FAKE, FAKE, None) == SHAPE
        for square in (0, 1):
            assert lib.if4_fp8_quantize_t(FAKE, dt, 16, 1 << 31, 1 << 31, square, FAKE, FAKE, None) == SHAPE
    for m, n, square in ((1, 1 << 27, 0), (1, 1 << 27, 1), (17, 1 << 31, 0), (1 << 31, 1 << 31, 0)):
        for dt in (BF16, F32):
            assert lib.if4_fp8_gemm(FAKE, FAKE, FAKE, FAKE, square, m, n, 16, FAKE, dt, n, None, 0, None) == SHAPE, (m, n)


def test_norm_and_rotation(lib):
    from adaptive_block_scaled_amd import qk
    for tokens in (1 << 26, (1 << 26) + 8, 1 << 31):
        a = qk._Args(table=FAKE, positions=FAKE, tokens=tokens, head_dim=64, rotary=64, table_rows=10, eps=1e-6, dtype=0,
                     out_dtype=1)
        for p in (a.q, a.k):
            p.x = p.y = p.weight = FAKE
            p.x_stride_token = p.y_stride_token = p.x_stride_head = p.y_stride_head = 64
        a.q.heads = 1
        assert lib.if4_norm_rotate(a, None) == SHAPE


def test_cache_and_attention(lib):
    from test_kv_abi import args, cache
    from adaptive_block_scaled_amd import kv_cache as kvc
    c = cache(kvc)
    assert lib.if4_kv_append(c, FAKE, FAKE, 1, 1 << 32, 64, 64, 64, 64, FAKE, 0, None) == SHAPE
    assert lib.if4_kv_read(c, FAKE, 1 << 32, FAKE, FAKE, 1, None) == SHAPE
    many = args(kvc, batch=1 << 25, total_q=1 << 25, max_q=1)
    assert lib.if4_kv_attention(c, many, FAKE, 1 << 50, None) == SHAPE


def test_eviction(lib):
    from test_kv_abi import args, cache
    from test_kv_evict_abi import mass
    from adaptive_block_scaled_amd import kv_cache as kvc, kv_evict as ev
    c, pool = cache(kvc), mass(ev, rows=FAKE)
    for kw in (dict(batch=1 << 25, total_q=1 << 25, max_q=1), dict(batch=1 << 15, total_q=1 << 22, max_q=1 << 22)):
        assert lib.if4_kv_weights(c, args(kvc, **kw), pool, FAKE, 1 << 50, None) == SHAPE, kw
    # lengths do not matter: a workgroup goes on to the keys that no other one has
    few, long = (args(kvc, batch=1 << 20, total_q=1 << 20, max_q=64, max_len=n) for n in (1 << 10, 1 << 29))
    assert lib.if4_kv_weights_workspace(c, long) <= 64 * lib.if4_kv_weights_workspace(c, few)
    assert lib.if4_kv_select(pool, FAKE, 1 << 22, 1, 10, 0, 0, FAKE, None, 0, None) == SHAPE
    assert lib.if4_kv_compact(c, FAKE, 5, FAKE, 1, 1 << 28, FAKE, 5, None) == SHAPE
