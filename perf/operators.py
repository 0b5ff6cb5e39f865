"""Cases of the paged IF4 KV cache: writing it, reading it back, and attention over it.

`run` computes each operator in its plain form (elementary torch operations) or, where `own` is true, through
`adaptive_block_scaled_amd.kv_cache`.

The cache (uint8 tensors; `pages` pages of `page_size` tokens, a multiple of 16; groups of 16 along the head dim D):
  k_codes  [pages, kv_heads, page_size, D/2]            rows as if4.quantize writes them
  k_scales [pages, kv_heads, page_size, D/16]
  v_codes  [pages, kv_heads, page_size/16, 16, 16, D/32]  (tile of 16 tokens, piece of D/16 dims, token, bytes)
  v_scales [pages, kv_heads, page_size/16, D/16, 16]      (tile, group, token)
A slot is page * page_size + offset.  IF4 itself (scale, both encodings, the choice, the bytes) is defined in include/if4.h.
"""
import functools
import math
import random

import numpy as np
import torch

own = False

GROUP = 16
DEVICE = "cuda"


# ---------------------------------------------------------------------------------------------------------------------
# Cases

def _attn(name, batch, q_lo, q_hi, ctx_lo, ctx_hi, heads, kv_heads, dim, page, window=0, sinks=0):
    return dict(name=name, op="attention", batch=batch, q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, heads=heads,
                kv_heads=kv_heads, dim=dim, page=page, window=window, sinks=sinks)


def listed():
    return [
        # one new token of each of 64 sequences goes into the cache after a decode step's projections
        dict(name="append_decode", op="append", tokens=64, kv_heads=8, dim=128, page=16, dtype="bf16"),
        # a long prompt's K and V, column slices of one fused QKV product, written and read back for a dense prefill
        dict(name="append_prompt", op="append", tokens=8192, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # an fp32 model with narrow heads and an odd number of tokens
        dict(name="append_odd_f32", op="append", tokens=1021, kv_heads=3, dim=64, page=32, dtype="f32"),
        # a whole 32k context leaves the cache in bf16 (moved to another format, or inspected)
        dict(name="read_context", op="read", tokens=32768, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # a short prefix in fp32, wide heads
        dict(name="read_prefix_f32", op="read", tokens=777, kv_heads=2, dim=256, page=16, dtype="f32"),
        # one user's next token: the latency of a single sequence
        _attn("decode_one", 1, 1, 1, 4097, 4097, 64, 8, 128, 16),
        # a serving batch's next tokens over contexts of mixed length
        _attn("decode_batch", 64, 1, 1, 3001, 12289, 64, 8, 128, 64),
        # few users with very long contexts
        _attn("decode_long", 4, 1, 1, 100003, 131071, 64, 8, 128, 128),
        # a chunk of a long prompt over what is already cached
        _attn("chunk_2k_of_16k", 1, 2048, 2048, 16384, 16384, 64, 8, 128, 64),
        # whole prompts, causal from their first token
        _attn("prompt_4k", 2, 4096, 4096, 4096, 4096, 64, 8, 128, 64),
        # narrow heads, a sliding window with four first tokens kept visible
        _attn("window_sinks", 3, 700, 1531, 9001, 20000, 32, 8, 64, 32, window=1024, sinks=4),
        # decodes and short chunks in one batch (scheduled together, or drafts to verify), wide heads, an odd head group
        _attn("mixed_wide", 24, 1, 61, 61, 5003, 21, 3, 256, 16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _at_most_listed(case, sizes, least):
    """The case with these sizes cut down together until it does no more work than the largest listed one of its operator."""
    tops = [work(c) for c in listed() if c["op"] == case["op"]]
    while any(work(case)[k] > max(t[k] for t in tops) for k in ("bytes", "flops")):
        case.update({n: max(least, case[n] * 4 // 5) for n in sizes})
    return case


def draw(rng):
    op = rng.choice(["append", "read", "attention", "attention", "attention", "attention"])
    dim = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128])
    if op != "attention":
        case = dict(op=op, tokens=_log_int(rng, 1, 8192 if op == "append" else 32768), kv_heads=rng.choice([1, 2, 3, 4, 8]), dim=dim,
                    page=page, dtype=rng.choice(["bf16", "bf16", "f32"]))
        return _at_most_listed(case, ["tokens"], 1)
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 7, 8])
    kind = rng.choice(["decode", "chunk", "mixed"])
    if kind == "decode":
        batch = _log_int(rng, 1, 64)
        hi = _log_int(rng, 16, 131072)
        q_lo = q_hi = 1
    elif kind == "chunk":
        batch = rng.choice([1, 1, 2, 3])
        q_hi = _log_int(rng, 64, 4096)
        q_lo = rng.randint(max(1, q_hi // 2), q_hi)
        hi = q_hi + _log_int(rng, 1, 16384)
    else:
        batch = _log_int(rng, 2, 32)
        q_lo, q_hi = 1, _log_int(rng, 2, 128)
        hi = q_hi + _log_int(rng, 16, 4096)
    lo = rng.randint(max(q_hi, hi // 4), hi)
    window, sinks = (_log_int(rng, 16, 4096), rng.choice([0, 1, 4, 64])) if rng.random() < 0.35 else (0, 0)
    case = _attn("", batch, q_lo, q_hi, lo, hi, heads, kv_heads, dim, page, window, sinks)
    del case["name"]
    return _at_most_listed(case, ["q_lo", "q_hi", "ctx_lo", "ctx_hi"], 1)


def _spread(lo, hi, n, step):
    """n whole numbers from lo to hi, both included where n > 1, in a mixed order that the case alone decides."""
    return [hi if n == 1 else lo + (hi - lo) * ((i * step) % n) // (n - 1) for i in range(n)]


def _lengths(case):
    b = case["batch"]
    odd = [s for s in (7, 11, 13) if math.gcd(s, b) == 1][0] if b > 1 else 1
    return _spread(case["q_lo"], case["q_hi"], b, 1), _spread(case["ctx_lo"], case["ctx_hi"], b, odd)


def _visible(case, q_len, ctx):
    """(row, key) pairs that attend, and the keys that any row sees, of one sequence (positions ctx - q_len .. ctx - 1)."""
    first, w, s = ctx - q_len, case["window"], case["sinks"]
    pos = np.arange(first, ctx, dtype=np.int64)
    if not w:
        return int((pos + 1).sum()), ctx
    start = np.maximum(0, pos - w + 1)
    return int((pos + 1 - start + np.minimum(s, start)).sum()), ctx - int(start[0]) + min(s, int(start[0]))


def work(case):
    d, kvh = case["dim"], case["kv_heads"]
    packed = d // 2 + d // GROUP
    if case["op"] != "attention":
        vectors, wide = 2 * case["tokens"] * kvh, d * (4 if case["dtype"] == "f32" else 2)
        # append: the inputs in, the cache bytes out, and (read back) in again and the values out
        once = vectors * (wide + packed) + 8 * case["tokens"]
        return {"bytes": 2 * once if case["op"] == "append" else once, "flops": 0}
    q_lens, ctxs = _lengths(case)
    seen = [_visible(case, q, c) for q, c in zip(q_lens, ctxs)]
    return {"bytes": 4 * sum(q_lens) * case["heads"] * d + 2 * kvh * packed * sum(k for _, k in seen),
            "flops": 4 * d * case["heads"] * sum(p for p, _ in seen)}


# ---------------------------------------------------------------------------------------------------------------------
# Inputs

def _vectors(gen, tokens, heads, dim, outliers):
    """Normal values; K has a few channels of a head that are much larger than the others, as trained models have."""
    x = torch.randn(tokens, heads, dim, generator=gen, device=DEVICE)
    if outliers:
        gain = torch.ones(heads, dim, device=DEVICE)
        gain.scatter_(1, torch.randint(0, dim, (heads, max(1, dim // 32)), generator=gen, device=DEVICE), 6.0)
        x *= gain
    return x


def _exponent(limit):
    """The cache's power of two: set beforehand for values up to `limit`, as a calibration does."""
    return math.ceil(math.log2(limit / (6.0 * 448.0)))


def _v_tiles(codes, scales):
    """V rows [pages, heads, page, ...] in the cache's order of V."""
    p, h, page, half = codes.shape
    c = codes.view(p, h, page // 16, 16, 16, half // 16).transpose(3, 4).contiguous()
    s = scales.view(p, h, page // 16, 16, half // 8).transpose(3, 4).contiguous()
    return c, s


def _filled_cache(gen, pages, page, kv_heads, dim, k_exp, v_exp):
    """A cache that holds K and V of tokens: rows of a pool of quantized tokens, each page's tokens drawn from it."""
    pool = min(4096, pages * page)
    k = _quantize(_vectors(gen, pool, kv_heads, dim, True).bfloat16(), k_exp)
    v = _quantize(_vectors(gen, pool, kv_heads, dim, False).bfloat16(), v_exp)
    at = torch.randint(0, pool, (pages, page), generator=gen, device=DEVICE)
    kc, ks = (t[at].transpose(1, 2).contiguous() for t in k)
    vc, vs = _v_tiles(*(t[at].transpose(1, 2).contiguous() for t in v))
    return {"k_codes": kc, "k_scales": ks, "v_codes": vc, "v_scales": vs}


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE).manual_seed(seed)
    kvh, dim, page = case["kv_heads"], case["dim"], case["page"]
    k_exp, v_exp = _exponent(48.0), _exponent(8.0)
    state = dict(op=case["op"], k_exp=k_exp, v_exp=v_exp, page=page)
    if case["op"] != "attention":
        n = case["tokens"]
        pages = -(-n // page) + 3
        # tokens fill the pages one after another; the pages come in any order
        order = torch.randperm(pages, generator=gen, device=DEVICE)
        at = torch.arange(n, device=DEVICE)
        state["slots"] = order[at // page] * page + at % page
        state["dtype"] = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        if case["op"] == "read":
            state["cache"] = _filled_cache(gen, pages, page, kvh, dim, k_exp, v_exp)
            return state
        # q, k and v as column slices of one product's rows
        fused = torch.cat([_vectors(gen, n, kvh, dim, False), _vectors(gen, n, kvh, dim, True), _vectors(gen, n, kvh, dim, False)], 1)
        fused = fused.to(state["dtype"])
        state["k"], state["v"] = fused[:, kvh:2 * kvh], fused[:, 2 * kvh:]
        state["cache"] = {name: torch.zeros(shape, dtype=torch.uint8, device=DEVICE) for name, shape in (
            ("k_codes", (pages, kvh, page, dim // 2)), ("k_scales", (pages, kvh, page, dim // GROUP)),
            ("v_codes", (pages, kvh, page // 16, 16, 16, dim // 32)), ("v_scales", (pages, kvh, page // 16, dim // GROUP, 16)))}
        return state
    q_lens, ctxs = _lengths(case)
    need = [-(-c // page) for c in ctxs]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=gen, device=DEVICE).to(torch.int32)
    table = torch.zeros(len(need), max(need), dtype=torch.int32, device=DEVICE)
    first = 0
    for b, m in enumerate(need):
        table[b, :m] = order[first:first + m]
        first += m
    total = sum(q_lens)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    state.update(
        q=_vectors(gen, total, case["heads"], dim, False).bfloat16(), cache=_filled_cache(gen, pages, page, kvh, dim, k_exp, v_exp),
        page_table=table, seq_lens=torch.tensor(ctxs, dtype=torch.int32, device=DEVICE),
        q_starts=torch.tensor(starts, dtype=torch.int32, device=DEVICE), max_q=max(q_lens), max_len=max(ctxs),
        scale=dim ** -0.5, window=case["window"], sinks=case["sinks"])
    return state


# ---------------------------------------------------------------------------------------------------------------------
# Plain forms

def _e4m3(code):
    e, m = (code >> 3).float(), (code & 7).float()
    value = torch.where(e > 0, torch.ldexp(1 + m / 8, e - 7), m * 2.0 ** -9)
    return torch.where(code == 127, torch.nan, value)


def _fma(a, b, c):
    """fp32 fma: the product is exact in 64 bits, and the sum is rounded to 32 once."""
    return (a.double() * b.double() + c.double()).float()


def _quantize(x, exp):
    """IF4 rows of x [..., D]: (codes [..., D/2], scales [..., D/16]).  The roundings are decided exactly: 32 bits hold what they
    need of bf16 inputs, fp32 inputs take 64."""
    wide = torch.float64 if x.dtype == torch.float32 else torch.float32
    g = x.to(wide).unflatten(-1, (-1, GROUP))
    a = g.abs()
    t = a.amax(-1) * 2.0 ** -exp / 6
    step = torch.exp2(torch.frexp(t)[1].to(wide) - 4).clamp(min=2.0 ** -9)
    sp = (torch.round(t / step) * step).clamp(max=448.0)
    zero, bad = sp == 0, ~torch.isfinite(t)
    s = torch.where(zero | bad, 1.0, sp).unsqueeze(-1) * 2.0 ** exp
    u = a / s
    half = torch.where(u < 2, 0.5, torch.where(u < 4, 1.0, 2.0))
    c = (torch.round(u / half) * half).clamp(max=6.0)
    q = torch.round(7 * a / (6 * s)).clamp(max=7.0)
    df, di = (_fma(a.double(), torch.tensor(7.0, device=x.device), -m.double() * k * s.double()) for m, k in ((c, 7), (q, 6)))
    start = torch.zeros_like(df[..., 0])
    ef, ei = (functools.reduce(lambda e, d: _fma(d, d, e), part.unbind(-1), start) for part in (df, di))
    pick = (ei < ef).unsqueeze(-1)
    index = torch.where(c < 2, 2 * c, torch.where(c < 4, c + 2, c / 2 + 4))
    nib = torch.where(pick, q, index).to(torch.uint8) + 8 * torch.signbit(g).to(torch.uint8)
    nib = torch.where((zero | bad).unsqueeze(-1), 0, nib).flatten(-2)
    f, e = torch.frexp(sp)
    byte = torch.where(sp < 2.0 ** -6, sp * 512, (e + 6) * 8 + (f * 16 - 8)).nan_to_num(0).to(torch.uint8) + 128 * pick.squeeze(-1).to(torch.uint8)
    byte = torch.where(bad, 127, torch.where(zero, 0, byte)).to(torch.uint8)
    return nib[..., 0::2] + 16 * nib[..., 1::2], byte


def _dequantize(codes, scales, exp):
    """fp32 values of IF4 rows: codes [..., D/2], scales [..., D/16]."""
    nib = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (-1, GROUP))
    m = (nib & 7).float()
    fp4 = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    sp = _e4m3(scales.int() & 127).unsqueeze(-1)
    y = torch.where((scales >= 128).unsqueeze(-1), 6 * m * sp / 7, fp4 * sp) * 2.0 ** exp
    return torch.where(nib >= 8, -y, y).flatten(-2)


def _rows_of_v(cache):
    """V's codes and scales as rows [pages, heads, page, ...]."""
    c, s = cache["v_codes"], cache["v_scales"]
    return c.transpose(3, 4).flatten(4).flatten(2, 3), s.transpose(3, 4).flatten(2, 3)


def _plain_read(state):
    page, slots, c = state["page"], state["slots"], state["cache"]
    vc, vs = _rows_of_v(c)
    p, o = slots // page, slots % page
    k = _dequantize(c["k_codes"][p, :, o], c["k_scales"][p, :, o], state["k_exp"])
    v = _dequantize(vc[p, :, o], vs[p, :, o], state["v_exp"])
    return k.to(state["dtype"]), v.to(state["dtype"])


def _plain_append(state):
    page, slots, c = state["page"], state["slots"], state["cache"]
    p, o = slots // page, slots % page
    c["k_codes"][p, :, o], c["k_scales"][p, :, o] = _quantize(state["k"], state["k_exp"])
    codes, scales = _quantize(state["v"], state["v_exp"])
    c["v_codes"][p, :, o // 16, :, o % 16] = codes.unflatten(-1, (16, -1))
    c["v_scales"][p, :, o // 16, :, o % 16] = scales


def _plain_attention(state):
    q, c, starts, lens = state["q"], state["cache"], state["q_starts"].long(), state["seq_lens"].long()
    table, max_q, n = state["page_table"].long(), state["max_q"], state["max_len"]
    total, heads, dim = q.shape
    batch, kvh = len(lens), c["k_codes"].shape[1]
    vc, vs = _rows_of_v(c)
    dense = lambda t: t[table].transpose(1, 2).flatten(2, 3)[:, :, :n]  # noqa: E731  [batch, kv_heads, n, ...]
    k = _dequantize(dense(c["k_codes"]), dense(c["k_scales"]), state["k_exp"])
    v = _dequantize(dense(vc), dense(vs), state["v_exp"])
    i, j = torch.arange(max_q, device=q.device), torch.arange(n, device=q.device)
    q_lens = starts[1:] - starts[:-1]
    rows = (starts[:-1, None] + i).clamp(max=total - 1)
    padded = q.float()[rows].unflatten(2, (kvh, -1)).permute(0, 2, 3, 1, 4).flatten(2, 3)  # [batch, kv_heads, group * max_q, D]
    s = torch.matmul(padded, k.transpose(2, 3).contiguous()).mul_(state["scale"]).unflatten(2, (-1, max_q))
    pos = (lens - q_lens)[:, None, None] + i[:, None]
    seen = j <= pos
    if state["window"]:
        seen &= (j > pos - state["window"]) | (j < state["sinks"])
    seen = seen[:, None, None]
    s = s.masked_fill_(~seen, -torch.inf)
    e = s.sub_(s.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    out = torch.matmul(e.flatten(2, 3), v).unflatten(2, (-1, max_q)) / e.sum(-1, keepdim=True).clamp(min=1e-30)
    out = out.permute(0, 3, 1, 2, 4).flatten(2, 3)  # [batch, max_q, heads, D]
    token = torch.arange(total, device=q.device)
    b = torch.searchsorted(starts, token, right=True) - 1
    return out[b, token - starts[b]].bfloat16()


def run(state):
    if own:
        from adaptive_block_scaled_amd import kv_cache
        cache = kv_cache.KVCache(**state["cache"])
        exps = dict(k_exp=state["k_exp"], v_exp=state["v_exp"])
        if state["op"] == "attention":
            return kv_cache.attention(state["q"], cache, state["page_table"], state["seq_lens"], state["q_starts"], max_q=state["max_q"],
                                      max_len=state["max_len"], scale=state["scale"], window=state["window"], sinks=state["sinks"], **exps)
        if state["op"] == "append":
            kv_cache.append(cache, state["k"], state["v"], state["slots"], **exps)
        return kv_cache.read(cache, state["slots"], dtype=state["dtype"], **exps)
    if state["op"] == "attention":
        return _plain_attention(state)
    if state["op"] == "append":
        _plain_append(state)
    return _plain_read(state)


# ---------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits

_E4M3 = [m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127]
_FP4 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
_INT4 = [6 * i / 7 for i in range(8)]


def _nearest(x, grid):
    """Index of the grid value nearest to x >= 0, an exact middle going to the even index."""
    mid = [(a + b) / 2 for a, b in zip(grid, grid[1:])]
    up = torch.bucketize(x, torch.tensor(mid, dtype=torch.float64, device=x.device), right=True)     # a middle goes up
    down = torch.bucketize(x, torch.tensor(mid, dtype=torch.float64, device=x.device), right=False)  # a middle goes down
    return torch.where(up % 2 == 0, up, down)


def _exact_round_trip(x, exp):
    g = x.double().reshape(*x.shape[:-1], -1, GROUP) / 2.0 ** exp
    table = lambda t: torch.tensor(t, dtype=torch.float64, device=x.device)  # noqa: E731
    s = table(_E4M3)[_nearest(g.abs().amax(-1, keepdim=True), [6 * v for v in _E4M3])]
    u = torch.where(s > 0, g.abs() / s, 0.0)
    f = table(_FP4)[_nearest(u, _FP4)]
    i = table(_INT4)[_nearest(7 * u, [6.0 * k for k in range(8)])]
    better = ((i - u) ** 2).sum(-1, keepdim=True) < ((f - u) ** 2).sum(-1, keepdim=True)
    return (torch.where(better, i, f) * s * torch.sign(g) * 2.0 ** exp).reshape(x.shape)


def _exact_rows(codes, scales, exp):
    """64-bit values of IF4 rows, by tables of every byte."""
    table = torch.tensor(_E4M3 + [math.nan], dtype=torch.float64, device=codes.device)
    both = torch.tensor([_FP4 + [-v for v in _FP4], _INT4 + [-v for v in _INT4]], dtype=torch.float64, device=codes.device)
    kind, s = (scales.long() >> 7).repeat_interleave(GROUP, -1), table[scales.long() & 127].repeat_interleave(GROUP, -1)
    nib = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.long, device=codes.device)
    nib[..., 0::2], nib[..., 1::2] = codes & 15, codes >> 4
    return both[kind, nib] * s * 2.0 ** exp


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "append":
        return tuple(_exact_round_trip(state[n], state[n + "_exp"]) for n in "kv")
    c, page = state["cache"], case["page"]
    kvh, dim = case["kv_heads"], case["dim"]

    def rows(slots, head):
        """K and V of these slots and this head, token by token."""
        p, o = slots // page, slots % page
        k = _exact_rows(c["k_codes"][p, head, o], c["k_scales"][p, head, o], state["k_exp"])
        v = _exact_rows(c["v_codes"][p, head, o // 16, :, o % 16].reshape(len(slots), dim // 2),
                        c["v_scales"][p, head, o // 16, :, o % 16], state["v_exp"])
        return k, v

    if case["op"] == "read":
        heads = [rows(state["slots"], h) for h in range(kvh)]
        return tuple(torch.stack([h[i] for h in heads], 1) for i in (0, 1))
    if work(case)["flops"] > 2e12:
        return None
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device=DEVICE)
    group = case["heads"] // kvh
    first = 0
    for b, (q_len, ctx) in enumerate(zip(*_lengths(case))):
        key = torch.arange(ctx, device=DEVICE)
        slots = state["page_table"][b].long()[key // page] * page + key % page
        for h in range(kvh):
            k, v = rows(slots, h)
            for r in range(0, q_len, 512):
                n = min(512, q_len - r)
                pos = ctx - q_len + r + torch.arange(n, device=DEVICE)[:, None]
                hidden = key > pos
                if case["window"]:
                    hidden |= (key <= pos - case["window"]) & (key >= case["sinks"])
                at = slice(first + r, first + r + n)
                for m in range(h * group, (h + 1) * group):
                    s = (state["q"][at, m].double() @ k.T) * state["scale"]
                    out[at, m] = torch.softmax(s.masked_fill(hidden, -math.inf), -1) @ v
        first += q_len
    return out
