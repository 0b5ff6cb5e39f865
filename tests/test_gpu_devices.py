"""Tensors of another device than the current one: a call runs on theirs.  Torch's default stream
is a null handle, which HIP takes as the current device's, so the binding makes the tensors'
device current for the time of a call."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def calls(device):
    """name: a call with preallocated outputs, which is marshalled in Python, and one without, in C++
    where there is one."""
    from adaptive_block_scaled_amd import fp8, if4, kv_cache as kvc, kv_evict as ev, qk
    g = torch.Generator(device=device).manual_seed(1)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device=device).bfloat16()

    def u8(*shape):
        return torch.zeros(*shape, dtype=torch.uint8, device=device)

    def i32(values):
        return torch.tensor(values, dtype=torch.int32, device=device)
    x, w = rand(32, 64), rand(48, 64)
    q4, w4 = if4.quantize(x), if4.quantize(w)
    q6, q8, w8 = if4.quantize_ifn(x, 6), fp8.quantize(x), fp8.quantize(w)
    q, k = rand(5, 4, 64), rand(5, 2, 64)
    norm = (*torch.ones(2, 64, device=device), qk.rotation_table(9, 64, device=device),
            torch.arange(5, device=device))
    cache = kvc.empty(4, 16, 2, 64, device)
    slots = torch.arange(5, device=device)
    kvc.append(cache, k, k, slots)
    table, lens, starts = i32([[0]]), i32([5]), i32([0, 5])
    batch = (q, cache, table, lens, starts)
    mass = torch.zeros(1, 2, 5, device=device)
    kept = ev.select(mass, lens, 3)

    def pair(call, *out):
        return lambda: call(out=out if len(out) > 1 else out[0]), lambda: call()
    return {
        "quantize": pair(lambda **o: if4.quantize(x, **o), u8(32, 32), u8(32, 4)),
        "quantize_t": pair(lambda **o: if4.quantize_t(x, **o), u8(64, 16), u8(64, 2)),
        "quantize_rht": pair(lambda **o: if4.quantize_rht(x, 3, **o), u8(32, 32), u8(32, 4)),
        "quantize_ifn": pair(lambda **o: if4.quantize_ifn(x, 6, **o), u8(32, 48), u8(32, 4)),
        "dequantize": pair(lambda **o: if4.dequantize(*q4, **o), torch.zeros(32, 64, device=device)),
        "dequantize_ifn": pair(lambda **o: if4.dequantize_ifn(*q6, 6, **o), torch.zeros(32, 64, device=device)),
        "gemm": pair(lambda **o: if4.gemm(*q4, 0, *w4, 0, **o), torch.zeros(32, 48, device=device)),
        "fp8.quantize": pair(lambda **o: fp8.quantize(x, **o), u8(32, 64), u8(32, 1)),
        "fp8.quantize_t": pair(lambda **o: fp8.quantize_t(x, **o), u8(64, 32), u8(64, 1)),
        "fp8.gemm": pair(lambda **o: fp8.gemm(*q8, *w8, **o), torch.zeros(32, 48, dtype=torch.bfloat16, device=device)),
        "norm_rotate": pair(lambda **o: qk.norm_rotate(q, k, *norm, **o), torch.zeros_like(q), torch.zeros_like(k)),
        "norm_rotate_backward": pair(lambda **o: qk.norm_rotate_backward(q, k, q, k, *norm, **o), torch.zeros_like(q),
                                     torch.zeros_like(k)),
        "read": pair(lambda **o: kvc.read(cache, slots, **o), torch.zeros_like(k), torch.zeros_like(k)),
        "attention": pair(lambda **o: kvc.attention(*batch, max_q=5, **o), torch.zeros_like(q)),
        "accumulate": (lambda: ev.accumulate(mass, *batch, max_q=5, out=torch.zeros_like(mass),
                                             workspace=u8(ev.workspace_bytes(cache, total_q=5, heads=4, batch=1, max_q=5,
                                                                             max_len=16))),
                       lambda: ev.accumulate(mass, *batch, max_q=5, out=torch.zeros_like(mass))),
        "select": pair(lambda **o: ev.select(mass, lens, 3, **o), torch.zeros_like(kept)),
        "compact": (lambda: ev.compact(kvc.KVCache(*(t.clone() for t in cache)), table, kept, i32([[2]])),) * 2,
    }


def flat(result):
    return list(result) if isinstance(result, tuple) else [result]


def test_the_tensors_device_is_made_current(monkeypatch):
    # as if another device were current: calls marshalled in Python change to the tensors' own
    entered = []

    class Device(torch.cuda.device):
        def __init__(self, device):
            entered.append(device)
            super().__init__(device)
    pairs = calls("cuda:0")
    for name, (own, plain) in pairs.items():
        want = flat(plain())
        if name == "compact":  # (marshalled in Python only where something is out of order)
            continue
        with monkeypatch.context() as m:
            m.setattr(torch.cuda, "device", Device)
            m.setattr(torch._C, "_cuda_getDevice", lambda: 5)
            del entered[:]
            got = flat(own())
        assert entered == [0], name
        assert all(torch.equal(a, b) for a, b in zip(got, want)), name


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="one device")
def test_tensors_of_the_second_device():
    for name, first, second in ((n, a, b) for (n, a), b in zip(calls("cuda:0").items(), calls("cuda:1").values())):
        want = flat(first[1]())
        for call in second:
            got = flat(call())
            torch.cuda.synchronize(1)
            assert torch.cuda.current_device() == 0
            assert all(a.device.index == 1 and torch.equal(a.cpu(), b.cpu()) for a, b in zip(got, want)), name
