"""Arguments of the KV cache's Python calls that are out of order in ways that
the kernels' own tests do not meet: each is an error that says so."""
import pytest

from test_gpu_kv_attention import kvc  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def test_a_cache_without_heads(kvc):
    cache = kvc.KVCache(*(torch.zeros(shape, dtype=torch.uint8, device="cuda")
                          for shape in kvc._shapes(2, 16, 0, 64)))
    slots = torch.arange(3, device="cuda")
    x = torch.zeros(3, 0, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: kvc.append(cache, x, x, slots), lambda: kvc.read(cache, slots),
                 lambda: kvc.attention(q, cache, i32(0, 1)[None], i32(3), i32(0, 3), max_q=3),
                 lambda: kvc.workspace_bytes(cache, total_q=3, heads=4, batch=1, max_q=3, max_len=3)):
        with pytest.raises(ValueError, match="kv_heads"):
            call()


def test_integers_beyond_what_the_c_calls_take(kvc):
    from adaptive_block_scaled_amd.if4 import IF4Error
    cache = kvc.empty(4, 16, 2, 64)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(40, 2, 64, generator=g).bfloat16().cuda()
    slots = torch.arange(40, device="cuda")
    kvc.append(cache, x, x, slots, -6, -6)
    out = (torch.empty_like(x), torch.empty_like(x))
    q = torch.randn(3, 4, 64, generator=g).bfloat16().cuda()

    def attend(**kw):
        kw = {**dict(max_q=3, k_exp=-6, v_exp=-6), **kw}
        return kvc.attention(q, cache, i32(0, 1, 2)[None], i32(40), i32(0, 3), **kw)

    for exp in (1 << 32, -6 - (1 << 32), 1 << 70):
        for call in (lambda: kvc.append(cache, x, x, slots, exp, 0), lambda: kvc.append(cache, x, x, slots, 0, exp),
                     lambda: kvc.read(cache, slots, exp, 0), lambda: kvc.read(cache, slots, 0, exp, out=out),
                     lambda: attend(k_exp=exp), lambda: attend(v_exp=exp)):
            with pytest.raises(IF4Error, match="exponent"):
                call()
    with pytest.raises(IF4Error):
        kvc.append(cache, x, x, slots, mode=1 << 32)
    for huge in (1 << 64, (1 << 64) + 5):
        assert torch.equal(attend(max_q=huge), attend(max_q=3))
        assert torch.equal(attend(max_len=huge), attend(max_len=1 << 40))
        assert torch.equal(attend(window=2, sinks=huge), attend(window=2, sinks=1 << 40))
        with pytest.raises(IF4Error, match="bad shape"):
            attend(max_q=-huge)
        sizes = dict(total_q=3, heads=4, batch=1)
        assert kvc.workspace_bytes(cache, max_q=huge, max_len=huge, **sizes) == \
            kvc.workspace_bytes(cache, max_q=3, max_len=1 << 40, **sizes)
