"""Which rows of `out` attention over the KV cache writes: those of a sequence,
up to max_q of each, and no others, however the work is split."""
import numpy as np
import pytest

from test_gpu_kv_attention import Batch, kvc  # noqa: F401  (kvc: the module's fixture)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

KEPT = 0x4321  # bf16 bits that no row of these calls can get

BATCHES = [  # heads, kv_heads, chunks, max_q
    (8, 1, [3, 1, 2], 2),                       # tiles of few rows
    (24, 1, [2, 1, 0], 1),
    (8, 1, [16, 3, 11], 9),                     # 33 to 128 rows
    (8, 2, [150, 3, 90], 100),                  # prompts
    (8, 2, [1, 1, 1, 1, 2, 1, 1, 150, 1], 120),  # single tokens beside a long chunk
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads,chunks,max_q", BATCHES)
def test_rows_without_a_sequence_and_past_max_q_are_left_alone(kvc, dim, heads, kv_heads, chunks, max_q):
    # a padded batch: rows before the first sequence and behind the last one, and a
    # chunk with more rows than max_q says
    lens = [2100, 700, 900, 1, 64, 333, 40, 1700, 500][:len(chunks)]
    b = Batch(kvc, lens, chunks, heads, kv_heads, dim, 16, 21)
    want, bound = b.reference()
    before, behind, total = 3, 5, int(b.starts[-1])
    q = torch.cat([torch.ones(before, heads, dim), b.q.float(), torch.ones(behind, heads, dim)]).bfloat16().cuda()
    table, seq_lens, starts = b.device()
    owned = np.zeros(before + total + behind, bool)
    for s, n in zip(b.starts, chunks):
        owned[before + s:before + s + min(n, max_q)] = True
    for max_len in (1, 2100, 100000):
        out = torch.full(q.shape, KEPT, dtype=torch.int16, device="cuda").view(torch.bfloat16)
        kvc.attention(q, b.cache, table, seq_lens, starts + before, max_q=max_q, max_len=max_len, out=out, **b.exps)
        bits = out.view(torch.int16).cpu().numpy()
        assert (bits[~owned] == KEPT).all(), (max_len, np.flatnonzero((bits != KEPT).any((1, 2)) & ~owned))
        got = out.cpu().double().numpy()[before:before + total][owned[before:before + total]]
        mine = owned[before:before + total]
        assert (np.abs(got - want[mine]) <= bound[mine]).all(), max_len
