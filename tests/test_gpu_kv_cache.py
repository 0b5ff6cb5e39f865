"""Writing the paged IF4 KV cache and reading it back, against the CPU oracle:
codes, scale bytes and values are equal bit for bit, and nothing else in the
cache changes."""
import numpy as np
import pytest

import kv_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvc():
    from adaptive_block_scaled_amd import kv_cache
    return kv_cache


def inputs(tokens, heads, dim, dtype, seed, spread=2.0):
    """Normal values times a log-normal factor per (token, head), a zero group,
    a group of zeros of both signs."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, heads, dim, generator=g)
    x *= torch.exp(spread * torch.randn(tokens, heads, 1, generator=g))
    if tokens:
        x[0, 0, :16] = 0.0
        x[-1, -1, 16:32] = torch.tensor([0.0, -0.0] * 8)
    return x.to(dtype)


def host(cache):
    return {n: t.cpu().numpy() for n, t in cache._asdict().items()}


def some_slots(n, total, seed):
    return torch.from_numpy(np.random.default_rng(seed).permutation(total)[:n].astype(np.int64))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,kv_heads,page,exps,mode", [
    (1, 1, 16, (0, 0), 0),
    (33, 3, 48, (-5, 2), 0),
    (157, 8, 64, (-60, 60), 1),
    (64, 2, 16, (3, -8), 2),
])
def test_append_is_the_quantize_of_the_library(kvc, oracle_mod, dim, dtype, tokens, kv_heads, page,
                                               exps, mode):
    pages = tokens // page + 3
    k, v = (inputs(tokens, kv_heads, dim, dtype, 10 + i) * 2.0 ** exps[i] for i in (0, 1))
    slots = some_slots(tokens, pages * page, 5)
    cache = kvc.empty(pages, page, kv_heads, dim)
    for t in cache:
        t.fill_(0xA5)
    kvc.append(cache, k.cuda(), v.cuda(), slots.cuda(), *exps, mode=mode)
    got = host(cache)
    untouched = np.setdiff1d(np.arange(pages * page), slots.numpy())
    for part, x, e in (("k", k, exps[0]), ("v", v, exps[1])):
        codes, scales = oracle_mod.quantize(x.float().numpy().reshape(-1, dim), e, mode=mode)
        codes, scales = codes.reshape(tokens, kv_heads, -1), scales.reshape(tokens, kv_heads, -1)
        for t in range(tokens):
            c, s = ref.slot_rows(got, part, int(slots[t]))
            assert np.array_equal(c, codes[t]) and np.array_equal(s, scales[t]), (part, t)
        for slot in untouched:
            c, s = ref.slot_rows(got, part, int(slot))
            assert (c == 0xA5).all() and (s == 0xA5).all(), (part, slot)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tokens,kv_heads,page,exps", [(1, 1, 16, (0, 0)), (99, 5, 80, (-6, 7))])
def test_read_gives_the_dequantized_values(kvc, oracle_mod, dim, dtype, tokens, kv_heads, page, exps):
    # any bytes: every nibble and scale byte, NaN scales among them
    pages = tokens // page + 2
    g = torch.Generator().manual_seed(3)
    cache = kvc.empty(pages, page, kv_heads, dim)
    for t in cache:
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    slots = some_slots(tokens, pages * page, 6)
    got = kvc.read(cache, slots.cuda(), *exps, dtype=dtype)
    bytes_ = host(cache)
    for part, y, e in zip("kv", got, exps):
        assert y.shape == (tokens, kv_heads, dim) and y.dtype == dtype
        rows = [ref.slot_rows(bytes_, part, int(s)) for s in slots]
        codes = np.concatenate([r[0] for r in rows])
        scales = np.concatenate([r[1] for r in rows])
        want = torch.from_numpy(oracle_mod.dequantize(codes, scales, e)).to(dtype)
        assert torch.equal(y.cpu().reshape(-1, dim).view(torch.uint8)[~torch.isnan(want).repeat_interleave(
            want.element_size(), 1)], want.view(torch.uint8)[~torch.isnan(want).repeat_interleave(
                want.element_size(), 1)])
        assert torch.equal(torch.isnan(y.cpu().reshape(-1, dim)), torch.isnan(want))


def test_round_trip_of_non_finite_values(kvc):
    x = inputs(20, 2, 128, torch.bfloat16, 1)
    x[3, 1, 5] = float("nan")
    x[4, 0, 127] = float("-inf")
    cache = kvc.empty(2, 16, 2, 128)
    slots = some_slots(20, 32, 1).cuda()
    kvc.append(cache, x.cuda(), x.cuda(), slots)
    for y in kvc.read(cache, slots, dtype=torch.float32):
        nan = torch.isnan(y.cpu())
        want = torch.zeros_like(nan)
        want[3, 1, :16] = True
        want[4, 0, 112:] = True
        assert torch.equal(nan, want)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_slots_outside_the_cache(kvc, dim):
    cache = kvc.empty(2, 32, 3, dim)
    x = inputs(6, 3, dim, torch.bfloat16, 2, spread=0.0).cuda()
    slots = torch.tensor([5, -1, 64, 63, -(1 << 40), 1 << 40], device="cuda")
    kvc.append(cache, x, x, slots)
    k, v = kvc.read(cache, slots)
    assert bool((k[[1, 2, 4, 5]] == 0).all()) and bool((v[[1, 2, 4, 5]] == 0).all())
    assert bool((k[[0, 3]] != 0).any(-1).all()) and torch.equal(k, v)
    used = torch.zeros(64, dtype=torch.bool)
    used[[5, 63]] = True
    every = torch.arange(64, device="cuda")
    rest = kvc.read(cache, every)
    for y in rest:
        assert bool((y.cpu()[~used] == 0).all())


def test_no_tokens(kvc):
    cache = kvc.empty(1, 16, 2, 64)
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    x = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    kvc.append(cache, x, x, none)
    k, v = kvc.read(cache, none)
    assert k.shape == v.shape == (0, 2, 64)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_slices_of_a_fused_projection(kvc, dtype):
    # k and v as column slices, heads in another order of strides, another stream
    n, h, dim = 45, 4, 64
    fused = inputs(n, 3 * h, dim, dtype, 4).cuda()
    k, v = fused[:, h:2 * h], fused.transpose(0, 1).contiguous().transpose(0, 1)[:, 2 * h:]
    slots = some_slots(n, 96, 2).cuda()
    want = kvc.append(kvc.empty(3, 32, h, dim), k.contiguous(), v.contiguous(), slots)
    cache = kvc.empty(3, 32, h, dim)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kvc.append(cache, k, v, slots)
        got = kvc.read(cache, slots)
    side.synchronize()
    for a, b in zip(cache, want):
        assert torch.equal(a, b)
    out = tuple(torch.full((n, h, dim), 7.0, device="cuda") for _ in range(2))
    kvc.read(cache, slots, dtype=None, out=out)
    for a, b in zip(got, out):
        assert torch.equal(a, b.bfloat16())


def test_offsets_beyond_32_bits(kvc):
    # over 4 GiB of codes for K and for V: the last pages, and a page whose
    # offset is just past 2^32
    dim, heads, page = 256, 8, 64
    pages = (1 << 32) // (heads * page * dim // 2) + 3
    cache = kvc.empty(pages, page, heads, dim)
    x = inputs(6, heads, dim, torch.bfloat16, 5).cuda()
    slots = torch.tensor([0, (pages - 3) * page, (pages - 3) * page + 1, (pages - 2) * page - 1,
                          pages * page - 1, page], device="cuda")
    kvc.append(cache, x, 2 * x, slots)
    small = kvc.empty(1, 16, heads, dim)
    at = torch.arange(6, device="cuda")
    kvc.append(small, x, 2 * x, at)
    for a, b in zip(kvc.read(cache, slots), kvc.read(small, at)):
        assert torch.equal(a, b)
    table = torch.tensor([[0], [pages - 3], [pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1, 2, 64], dtype=torch.int32, device="cuda")
    q = inputs(3, heads, dim, torch.bfloat16, 6, spread=0.0).cuda()
    starts = torch.arange(4, dtype=torch.int32, device="cuda")
    got = kvc.attention(q, cache, table, lens, starts, max_q=1, max_len=64)
    b = {n: torch.cat([t[:1], t[pages - 3:pages - 2], t[pages - 1:]]).cpu().numpy()
         for n, t in cache._asdict().items()}
    want, bound = ref.attention(q.cpu().double().numpy(), b, np.array([[0], [1], [2]]), [1, 2, 64],
                                [0, 1, 2, 3], dim ** -0.5, 0, 0)
    assert (np.abs(got.cpu().double().numpy() - want) <= bound).all()


def test_refusals_of_the_binding(kvc):
    cache = kvc.empty(2, 16, 2, 64)
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(3, device="cuda")
    bad = [  # what is wrong, the call's k, v, slots
        ("k", x[:, :1], x, slots), ("k", x[..., :32], x, slots), ("k", x[0], x, slots),
        ("v", x, x[:2], slots), ("v", x, x.float(), slots), ("v", x, x.cpu(), slots),
        ("stride", x.transpose(1, 2).contiguous().transpose(1, 2), x, slots),
        ("slots", x, x, slots[:2]), ("slots", x, x, slots.int()), ("slots", x, x, slots.cpu()),
        ("slots", x, x, torch.arange(6, device="cuda")[::2]),
    ]
    for what, k, v, s in bad:
        with pytest.raises(ValueError, match=what):
            kvc.append(cache, k, v, s)
    with pytest.raises(TypeError):
        kvc.append(cache, x.half(), x.half(), slots)
    from adaptive_block_scaled_amd.if4 import IF4Error
    with pytest.raises(IF4Error, match="misaligned"):
        odd = torch.zeros(3, 2, 68, dtype=torch.bfloat16, device="cuda")[..., :64]
        kvc.append(cache, odd, odd, slots)
    with pytest.raises(IF4Error, match="exponent"):
        kvc.append(cache, x, x, slots, k_exp=99)
    for what, change in (("v_codes", dict(v_codes=cache.v_codes[:1])),
                         ("k_scales", dict(k_scales=cache.k_scales.cpu())),
                         ("v_scales", dict(v_scales=cache.v_scales.int())),
                         ("k_codes", dict(k_codes=cache.k_codes[0])),
                         ("head_dim", dict(k_codes=cache.k_codes[..., :16]))):
        with pytest.raises(ValueError, match=what):
            kvc.read(cache._replace(**change), slots)
    with pytest.raises(ValueError, match="slots"):
        kvc.read(cache, slots[None])
    with pytest.raises(ValueError, match="v must"):
        kvc.read(cache, slots, out=(x, x[:2]))
    with pytest.raises(TypeError):
        kvc.read(cache, slots, dtype=torch.float16)
