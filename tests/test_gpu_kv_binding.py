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
