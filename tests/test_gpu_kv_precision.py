"""Attention over the KV cache where one key takes nearly all of a row: how the
many small probabilities of a long context count."""
import math

import pytest

from test_gpu_kv_attention import kvc  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

PAGE = 1024
# (heads of the one kv head, dim): one token's rows for the kernels of 16 and 32 rows, of up to
# 128, of prompts, and of wide heads
ROWS = [(1, 64), (32, 64), (40, 64), (150, 64), (8, 128), (24, 128), (60, 128), (130, 128), (8, 256), (40, 256)]


def one_large_key(kvc, keys, heads, dim, log2_p, first_v):
    """One token over `keys` keys, the first of which has a score that is log2_p (in powers of
    two) above all others'.  K is 6 in the first key and -6 in the others, V is 6 and
    in the first key `first_v`: FP4 codes 7 and 15 at scale 1, all exact."""
    cache = kvc.empty(keys // PAGE, PAGE, 1, dim)
    cache.k_codes.fill_(0xFF)
    cache.k_codes[0, 0, 0] = 0x77
    cache.k_scales.fill_(0x38)
    cache.v_codes.fill_(0x77)
    cache.v_scales.fill_(0x38)
    if first_v == 0:
        cache.v_codes[0, 0, 0, :, 0] = 0
    else:
        assert first_v == 6
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.ones(1, heads, dim, dtype=torch.bfloat16, device="cuda")
    scale = log2_p * math.log(2) / (12 * dim)
    # (a hint of one key: no splits, so that one running maximum meets as many keys as can be)
    return kvc.attention(q, cache, torch.arange(keys // PAGE, **i32)[None], torch.tensor([keys], **i32),
                         torch.tensor([0, 1], **i32), max_q=1, max_len=1, scale=scale).double()


@pytest.mark.parametrize("heads,dim", ROWS)
@pytest.mark.parametrize("log2_p", [20.6, 23.4, 24.5, 25.02])
def test_the_sum_is_that_of_the_rounded_probabilities(kvc, heads, dim, log2_p):
    # all values are 6, so every row is 6 whatever the probabilities are, if the sum that
    # it is divided by counts what the product with V counts.  What is left: sums in fp32
    # (at most 2^20 / 4 / 4 additions in a row, of 2^-25 of the sum on average: 2^-9 at the
    # worst) and the rounding to bf16 (2^-9)
    out = one_large_key(kvc, 1 << 20, heads, dim, log2_p, 6)
    assert float((out - 6).abs().max()) <= 6 * 2.0 ** -8


@pytest.mark.parametrize("heads,dim", [r for r in ROWS if r[0] <= 32])
@pytest.mark.parametrize("log2_p", [16.3, 20.6, 23.4, 24.5, 25.2])
def test_many_small_probabilities_count(kvc, heads, dim, log2_p):
    # the first key takes nearly all and has V = 0, so a row is what 131071 small
    # probabilities p make of V = 6.  In tiles of few rows probabilities carry 2^6 at the least
    # where the largest one is 1, so fp16 holds p 2^6 within 2^-25 (or 2^-11 of it, where it is not
    # subnormal); exp2 and its argument are within 2^-16 for scores of these sizes, the
    # output's rounding 2^-9
    keys = 1 << 17
    out = one_large_key(kvc, keys, heads, dim, log2_p, 0)
    p = (keys - 1) * 2.0 ** -log2_p
    want = 6 * p / (1 + p)
    far = max(2.0 ** (log2_p - 31), 2.0 ** -11) + 2.0 ** -9 + 2.0 ** -12
    assert float((out / want - 1).abs().max()) <= far


@pytest.mark.parametrize("heads,dim", ROWS)
@pytest.mark.parametrize("log2_score", [10, 20, 24, 26])
def test_scores_of_any_size_stay_finite(kvc, heads, dim, log2_score):
    # scores of +- 2^log2_score powers of two, whose fp32 spacing reaches 4: the keys that score highest
    # share a row, the others have nothing of it
    cache = kvc.empty(2, PAGE, 1, dim)
    cache.k_codes.fill_(0xFF)
    cache.k_codes[1, 0, 7::64] = 0x77
    cache.k_scales.fill_(0x38)
    cache.v_codes.fill_(0x77)
    cache.v_codes[1, 0, :, :, 7::8] = 0x55
    cache.v_scales.fill_(0x38)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.ones(1, heads, dim, dtype=torch.bfloat16, device="cuda")
    scale = 2.0 ** log2_score * math.log(2) / (6 * dim)
    for max_len in (1, 2 * PAGE):
        out = kvc.attention(q, cache, torch.arange(2, **i32)[None], torch.tensor([2 * PAGE], **i32),
                            torch.tensor([0, 1], **i32), max_q=1, max_len=max_len, scale=scale).double()
        # V: code 5 (3) in tokens 7, 15, .. of each tile, those of the keys 7, 71, .. among them
        assert float((out - 3).abs().max()) <= 3 * 2.0 ** -8


@pytest.mark.parametrize("heads,dim", ROWS)
def test_the_largest_probability_is_at_least_one(kvc, heads, dim):
    # scores rise once, by a little more than a whole number of powers of two, and what is
    # 2^-24.64 of the largest is left: half of the smallest fp16 number is 2^-25, so it
    # counts as something if the largest probability is held as 1 or more.
    # K: 64 keys with 13/16 of the dims at -6 and the rest at 6, one of 6, the others of -6;
    # V is 6 in the others only.  A probability is 2^-25 off at the most, the output 2^-9,
    # and the other roundings (exp2, sums of 2^16 / 16 additions, V's normaliser) 2^-10
    keys, log2_p = 1 << 16, 24.64
    cache = kvc.empty(keys // PAGE, PAGE, 1, dim)
    cache.k_codes.fill_(0xFF)
    cache.k_codes[0, 0, :64, :dim * 3 // 32] = 0x77
    cache.k_codes[0, 0, 64] = 0x77
    cache.k_scales.fill_(0x38)
    cache.v_codes.fill_(0x77)
    cache.v_codes[0, 0, :4] = 0
    cache.v_codes[0, 0, 4, :, 0] = 0
    cache.v_scales.fill_(0x38)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.ones(1, heads, dim, dtype=torch.bfloat16, device="cuda")
    scale = log2_p * math.log(2) / (12 * dim)
    out = kvc.attention(q, cache, torch.arange(keys // PAGE, **i32)[None], torch.tensor([keys], **i32),
                        torch.tensor([0, 1], **i32), max_q=1, max_len=1, scale=scale).double()
    rest = keys - 65
    whole = 1 + 64 * 2.0 ** (-log2_p * 13 / 16) + rest * 2.0 ** -log2_p
    want = 6 * rest * 2.0 ** -log2_p / whole
    far = 6 * rest * 2.0 ** -25 + want * (2.0 ** -9 + 2.0 ** -10)
    assert float((out - want).abs().max()) <= far
